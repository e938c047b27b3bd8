// kda_attn_fwd.cu -- causal softmax attention on the tensor cores (sm_103a): whole prompts
// of a packed batch (kda_attn_prefill) and chunks of new tokens over a paged cache
// (kda_attn_paged, sequences of more than kFewRows query rows).
//
// A block takes 256 query rows of one key head at a time.  A row is a (token, query head of
// the group) pair, token major, so that a group of any size fills the tiles and few tokens of a
// large group still make one.  The rows are two tiles of 128; keys and values pass
// through a ring of 128-key tiles in shared memory (TMA, 128-byte swizzle).  For each key
// tile and row tile
//
//   S = Q K^T               tcgen05, fp32 in tensor memory
//   P = 2^(c S - c m + u)   one thread a row: its 128 scores in registers, c = scale log2 e
//   O += P V                tcgen05, P 16 bits in tensor memory over the columns of S
//
// While one tile's softmax runs, the tensor cores work on the other's products.  m is the
// running maximum of the row.  O and the running sum are rescaled only when the maximum
// has grown by more than 2^8 (fp16: 2^4), which bf16 and fp32 have the range for: after the first tiles
// hardly ever, and it is the softmax threads themselves that do it, between the products.  fp16
// ends at 2^16 and has a fixed step of 2^-24 below 2^-14, so that u = 11 there (bf16: 0): P is at most
// 2^15, and the many small weights of a long prompt next to a large one are still there (with u = 0 what is
// below 2^-25 of the largest would be counted in the sum and be missing in O).  P is rounded to 16 bits because the tensor cores
// read it so (half a step of P's own value); sums, maxima and O are fp32.
//
// Keys that a row may not see get the score -inf by a select, and value rows behind a
// sequence's last key are cleared in shared memory before the product (0 * NaN is NaN).
//
// Prompts: a block a row tile, the longest of a sequence first.  (Blocks that stay and take the
// next row tile as they come, by cancelling launches, were no faster: 354 us against 350 us for
// 8192 tokens, 32 on 8 heads of 128.  These take 340 us by themselves and 360 in a row of calls; at the sustained
// rate of the card's own matrix product it would be 323 us.)  A row tile's keys are not cut here, so that prompts of few row
// tiles are as long as the longest: 8192 tokens take 93 us with one head, and 144 with 12 on one.
// Chunks over a cache: few row tiles and a long axis of keys, so that the keys of all row tiles are laid end to end and cut into as many
// equal runs as there are SMs (512 tokens behind 32k: 310 -> 203 us, with the registers and uniform values
// of the softmax warps taken in the same step); a warp finds the
// next piece of the block's run while the others are busy with this one, and a row tile that
// is cut leaves shares, which a second kernel joins.
//
// Registers: the softmax warps need their 128 scores and as much again, more than a
// 384-thread block gives each thread (168), so that the third warpgroup hands over its own: 345
// us for the 8192 tokens instead of 376 us, when that was tried.  One warp issues both tiles' products (two
// warps: 525 us), and P is handed over whole (in halves: 415 us).  The ring's depth counts
// up to four tiles (three: 450 us, four: 351 us, five: 350 us).
#include "kda_attn_plan.cuh"

using namespace kda;

namespace {

__device__ unsigned g_attn_status;

constexpr int kThreads = 384;      // two softmax warpgroups; products, loads, the search for work, one idle warp
constexpr int kProductWarp = 8, kLoadWarp = 9, kWorkWarp = 10;
constexpr int kTileRows = 256;
// log2 of the growth of a maximum that O is rescaled for, and of what weights are stored times (see the top)
template <bool BF16>
constexpr float kGrowth = BF16 ? 8.f : 4.f;
template <bool BF16>
constexpr float kUp = BF16 ? 0.f : 11.f;
// A sum of weights without that factor.
template <bool BF16>
__device__ __forceinline__ float plain_sum(float l) { return BF16 ? l : l * (1.f / 2048.f); }
constexpr int kSMs = 152;
constexpr int kRuns = 128;         // runs of sequences whose work is summed up

template <int D>
struct Lay {
    static constexpr int kTileBytes = kAttnKeys * D * 2;              // a tile of keys, values, or 128 queries
    static constexpr int kBlockBytes = kAttnKeys * 128;               // 64 channels of it
        static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes;
};

// A piece of work: query rows from tile * kTileRows on of sequence n (tokens [a, a + tokens),
// `keys` keys), one key head, key tiles [j0, j0 + n_of[i]) for row tile i.
struct Work {
    int32_t some, n, tile, head;
    int64_t a;
    int32_t tokens, keys, rows;    // rows of the sequence from this tile on
    int32_t j0, n_of[2];
    int32_t turn;                  // the walk begins with key tile j0 + turn, and j0 follows on the last
    int32_t slot;                  // where its share goes; -1: it is the whole
};

struct Control {
    uint64_t q_full[2][2], full[8], empty[8], s_full[2], p_ready[2], o_full[2], work_full[2], work_empty[2], done;
    uint32_t tmem;
    Work work[2];
    int64_t before[kRuns];         // units of work in front of each run of sequences
    int64_t scan[kThreads / 32];
};

// Shares of split row tiles, and what the joining kernel needs to know of them.
struct Shares {
    int32_t *rec;     // [records][4]
    float *lse;       // [slots][rows]
    float *out;       // [slots][rows][d]
};

// ---------------------------------------------------------------- the next piece of work
// Sequence that holds unit u of the batch: by the threads' sums, then within the run of one
// thread; `first`: its first unit.
template <typename Cost>
__device__ __forceinline__ int find_sequence(const Control &ct, int N, int64_t u, Cost cost, int64_t &first) {
    int lo = 0, hi = kRuns;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ct.before[mid] <= u) lo = mid; else hi = mid;
    }
    const int per = (N + kRuns - 1) / kRuns;
    int64_t at = ct.before[lo];
    for (int n = lo * per; n < min(N, lo * per + per); ++n) {
        const int64_t c = cost(n);
        if (u < at + c) {
            first = at;
            return n;
        }
        at += c;
    }
    first = at;
    return -1;
}

// What the roles need of a piece of work.
template <bool PAGED>
__device__ __forceinline__ void fill(Work &w, const Attn &A, const AttnSeq &sq, int n, int tile, int head) {
    w.some = 1;
    w.n = n;
    w.tile = tile;
    w.head = head;
    w.a = sq.a;
    w.tokens = (int32_t)(sq.b - sq.a);
    w.keys = (int32_t)sq.keys;
    w.rows = w.tokens * A.G - tile * kTileRows;
    w.slot = -1;
    w.j0 = 0;
    w.turn = 0;
}
// Key tiles that the rows of row tile i see.
__device__ __forceinline__ int32_t tiles_seen(const Work &w, int G, int i) {
    const int32_t last = min(w.rows, (i + 1) * 128) - 1;   // last row of the tile
    if (last < i * 128) return 0;
    const int32_t seen = w.keys - w.tokens + (w.tile * kTileRows + last) / G + 1;
    return (max(0, min(seen, w.keys)) + kAttnKeys - 1) / kAttnKeys;
}

// Chunks over a cache: the cost of a sequence's first t row tiles, in key tiles; two more a
// row tile for what it costs however few they are.
constexpr int kOver = 2;
struct Chunk {
    int32_t tiles;
    int64_t behind;
    int32_t G;
    __device__ __forceinline__ int64_t upto(int64_t t) const {
        return kOver * t + (t * behind + kTileRows / 2 * t * (t + 1) / G) / kAttnKeys;
    }
};
__device__ __forceinline__ Chunk chunk_of(const Attn &A, int n, int few) {
    const AttnSeq s = attn_seq<true>(A, n);
    const int64_t tokens = s.b - s.a, rows = tokens * A.G;
    return Chunk{rows > few ? (int32_t)((rows + kTileRows - 1) / kTileRows) : 0, s.keys > tokens ? s.keys - tokens : 0, A.G};
}

// Row number r of a sequence as (token, head of the group), walked without divisions.
struct Row {
    int tok, g;
    __device__ __forceinline__ Row(int r, int G) : tok(r / G), g(r - r / G * G) {}
    __device__ __forceinline__ void add(const Row &s, int G) {
        tok += s.tok;
        g += s.g;
        if (g >= G) g -= G, ++tok;
    }
};
__device__ __forceinline__ void cp_async16(uint32_t to, const void *from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

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
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = attn_warp();
    const int G = A.G;

    if (tid == 0) {
        sm100::prefetch_tmap(&kmap);
        sm100::prefetch_tmap(&vmap);
        for (int i = 0; i < NST; ++i) {
            sm100::mbar_init(&ct.full[i], 1);
            sm100::mbar_init(&ct.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(&ct.q_full[i][0], 128);
            sm100::mbar_init(&ct.q_full[i][1], 128);
            sm100::mbar_init(&ct.s_full[i], 1);
            sm100::mbar_init(&ct.p_ready[i], 128);
            sm100::mbar_init(&ct.o_full[i], 1);
            sm100::mbar_init(&ct.work_full[i], 1);
            sm100::mbar_init(&ct.work_empty[i], 10);
        }
        sm100::mbar_init(&ct.done, 1);
        sm100::fence_mbar_init();
    }
    if (warp == kProductWarp) {
        sm100::tmem_alloc(&ct.tmem, 512);
        sm100::tmem_relinquish();
    }
    // how much work there is in front of each run of sequences
    auto tiles_of = [&](int n) {   // prompts: a unit is a row tile
        const AttnSeq s = attn_seq<false>(A, n);
        return ((s.b - s.a) * G + kTileRows - 1) / kTileRows;
    };
    auto cost_of = [&](int n) {    // chunks
        const Chunk c = chunk_of(A, n, few);
        return c.upto(c.tiles);
    };
    const int same = PAGED || A.cu ? -1 : (int)((A.seq_len * G + kTileRows - 1) / kTileRows);
    const bool small = !PAGED && A.N <= 32;   // each warp forms the sums itself
    int64_t total = (int64_t)A.N * same;
    if ((PAGED || same < 0) && !small) {
        const int per = (A.N + kRuns - 1) / kRuns, lo = tid * per, hi = tid < kRuns ? min(A.N, lo + per) : 0;
        int64_t mine = 0;
        for (int n = lo; n < hi; ++n) mine += PAGED ? cost_of(n) : tiles_of(n);
        mine = block_scan<kThreads>(mine, total, ct.scan);
        if (tid < kRuns) ct.before[tid] = mine;
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = ct.tmem;
    bool ok = true;
    constexpr int kPieces = PAGED ? INT32_MAX : 1;
    // Piece k of the block's work; chunks: from the warp that finds them; prompts: the row tile of the
    // block's number.
    auto piece = [&](int k, Work &w) {
        if (PAGED) {
            ok = attn_wait_long(&ct.work_full[k & 1], (k / 2) & 1, &g_attn_status);
            if (ok) w = ct.work[k & 1];
            return ok && w.some;
        }
        const uint32_t head = blockIdx.x % (uint32_t)A.Hkv, tile = blockIdx.x / (uint32_t)A.Hkv;
        int n;
        int64_t first, at;
        if (same < 0 && small) {
            const int64_t tiles = lane < A.N ? tiles_of(lane) : 0, all = __shfl_sync(0xffffffffu, warp_scan(tiles), 31);
            if (tile >= all) return false;
            at = all - 1 - tile;
            n = warp_find(tiles, at, first);
        } else {
            if (tile >= total) return false;
            at = total - 1 - tile;
            if (same >= 0) {
                n = (int)((uint32_t)at / (uint32_t)same);
                first = (int64_t)n * same;
            } else {
                n = find_sequence(ct, A.N, at, tiles_of, first);
            }
        }
        fill<false>(w, A, attn_seq<false>(A, n), n, (int)(at - first), (int)head);
        w.n_of[0] = tiles_seen(w, G, 0);
        w.n_of[1] = tiles_seen(w, G, 1);
        return true;
    };
    // the piece's entry may be written again
    auto read = [&](int k) {
        if (!PAGED) return;
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&ct.work_empty[k & 1]);
    };

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (PAGED && warp == kWorkWarp) {
        // ------------------------------------------------ the next piece of work
        // units [u, end) of heads * total, the last piece first (see where turn is set)
        const int64_t all = total * A.Hkv;
        const int64_t blocks = max((int64_t)1, min((int64_t)gridDim.x, all / 8));
        auto edge = [&](int64_t b) { return all * b / blocks; };
        const int64_t run = max((int64_t)1, all / blocks);
        int64_t u = 0, end = 0;
        if (lane == 0) sh.rec[blockIdx.x * 4] = 0;
        if (blockIdx.x < blocks) u = edge(blockIdx.x), end = edge(blockIdx.x + 1);
        for (int k = 0;; ++k) {
            if (k >= 2) {
                ok = attn_wait_long(&ct.work_empty[k & 1], (k / 2 - 1) & 1, &g_attn_status);
            }
            Work w;
            w.some = 0;
            while (ok && u < end && !w.some) {
                const int64_t head = (end - 1) / total, in = end - 1 - head * total;
                int64_t first;
                const int n = find_sequence(ct, A.N, in, cost_of, first);
                if (n < 0) break;
                const Chunk c = chunk_of(A, n, few);
                int lo = 0, hi = c.tiles;   // row tile
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (first + c.upto(mid) <= in) lo = mid; else hi = mid;
                }
                // its units [t0, t1); an edge next to either end counts as that end
                const int64_t t0 = head * total + first + c.upto(lo), t1 = head * total + first + c.upto(lo + 1);
                auto snap = [&](int64_t x) { return x <= t0 + kOver + 1 ? t0 : x >= t1 - 2 ? t1 : x; };
                const int64_t from = u <= t0 ? t0 : snap(u), to = end >= t1 ? t1 : snap(end);
                end = t0;
                if (from >= to) continue;
                fill<true>(w, A, attn_seq<true>(A, n), n, lo, (int)head);
                const int32_t seen[2] = {tiles_seen(w, G, 0), tiles_seen(w, G, 1)};
                const int32_t most = max(seen[0], seen[1]);
                // edges inside: the first belongs to the block that begins the tile
                const int64_t b0 = ((t0 + kOver + 2) * blocks + all - 1) / all, b1 = ((t1 - 2) * blocks + all - 1) / all - 1;
                const int32_t splits = b1 >= b0 ? (int32_t)(b1 - b0) + 2 : 1;
                auto key = [&](int64_t x) {   // units of the tile before x -> key tiles
                    if (x >= t1) return most;
                    if (x <= t0 + kOver) return 0;
                    return (int32_t)((x - t0 - kOver) * most / (t1 - t0 - kOver));
                };
                w.j0 = key(from);
                const int32_t j1 = key(to);
                w.n_of[0] = max(0, min(seen[0], j1) - w.j0);
                w.n_of[1] = max(0, min(seen[1], j1) - w.j0);
                // The row tiles of a head read the same keys, each in blocks of their own: they should do so at
                // about the same time, or HBM delivers every key once a row tile.  So a block begins
                // with the piece that starts a row tile, and every piece with a multiple of the run
                // (512 tokens behind 32k: 960 -> 142 MB from HBM, 203 -> 183 us by itself; 195 in a row of calls).
                const int64_t begin = (w.j0 + run - 1) / run * run;
                const int32_t walk = max(w.n_of[0], w.n_of[1]);
                if (begin > w.j0 && begin < w.j0 + walk) {
                    w.turn = (int32_t)(begin - w.j0);
                    // (both row tiles walk all key tiles then: what they do not see is masked)
                    w.n_of[0] = walk;
                    w.n_of[1] = w.rows > 128 ? walk : 0;
                }
                if (splits > 1) {
                    const bool begins = from == t0;
                    w.slot = begins ? 2 * blockIdx.x + 1 : 2 * blockIdx.x;
                    if (begins && lane == 0) {
                        int32_t *rec = sh.rec + blockIdx.x * 4;
                        rec[1] = n;
                        rec[2] = lo;
                        rec[3] = (int32_t)head;
                        rec[0] = splits;
                    }
                }
            }
            if (lane == 0) {
                ct.work[k & 1] = w;
                sm100::mbar_arrive(&ct.work_full[k & 1]);
            }
            __syncwarp();
            if (!w.some) break;
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------ keys and values
        const int boxes = kAttnKeys / box;             // boxes of 64 channels that make a block
        const int mine = lane / boxes, which = lane % boxes;
        const bool issues = lane < boxes * (D / 64);
        uint32_t c = 0;   // tiles asked for
        bool bad = false;
        for (int k = 0; ok && k < kPieces; ++k) {
            Work w;
            if (!piece(k, w)) break;
            const int n = max(w.n_of[0], w.n_of[1]), j0 = w.j0, head = w.head, keys = w.keys, turn = w.turn;
            const int64_t a = w.a;
            const int32_t *row = PAGED ? A.table + (int64_t)w.n * A.wide : nullptr;
            if (PAGED) bad = bad || A.lens[w.n] > (int64_t)A.wide * A.page;
            read(k);
            for (int x = 0; x < 2 * n; ++x, ++c) {
                // order: K0, K1, V0, K2, V1, ...
                const bool last = x == 2 * n - 1, values = last || (x > 0 && (x & 1) == 0);
                int j = (values ? (last ? n - 1 : x / 2 - 1) : (x + 1) / 2) + turn;
                j = j0 + (j < n ? j : j - n);
                int page = 0, at;
                if (PAGED) {
                    const int64_t first = (int64_t)j * kAttnKeys + which * box;
                    page = A.P;   // past the cache: reads zeros
                    at = (int)(first % A.page);
                    if (issues && first < keys) {
                        const int p = row[first / A.page];
                        if (p >= 0 && p < A.P) page = p; else bad = true;
                    }
                } else {
                    at = (int)(a + (int64_t)j * kAttnKeys);
                }
                const uint32_t st = c % NST;
                if (c >= NST) ok = attn_wait(&ct.empty[st], (c / NST - 1) & 1, &g_attn_status);
                if (!ok) break;
                uint8_t *to = ring + st * L::kTileBytes;
                if (lane == 0) sm100::mbar_arrive_expect_tx(&ct.full[st], L::kTileBytes);
                __syncwarp();
                if (issues)
                    tma_load_4d(to + mine * L::kBlockBytes + which * box * 128, values ? &vmap : &kmap, &ct.full[st],
                                mine * 64, head, at, page);
            }
        }
        if (bad) atomicOr(&g_attn_status, kCacheBadPage);
        __syncwarp();
        // no copy may land after the block's end
        for (uint32_t x = c > NST ? c - NST : 0; x < c; ++x) attn_wait(&ct.full[x % NST], (x / NST) & 1, &g_attn_status);
    } else if (warp == kProductWarp) {
        // ------------------------------------------------ products
        const uint32_t q_at = sm100::smem_u32(Qs), ring_at = sm100::smem_u32(ring);
        auto wait = [&](uint64_t *bar, uint32_t parity) { return attn_wait(bar, parity, &g_attn_status); };
        auto full = [&](uint32_t c) { return wait(&ct.full[c % NST], (c / NST) & 1); };
        auto scores = [&](int i, uint32_t c) {
            mma_rows<D, BF16, 128>(tmem + i * 128, q_at + i * L::kTileBytes, ring_at + (c % NST) * L::kTileBytes,
                                   L::kBlockBytes, L::kBlockBytes);
            sm100::mma_commit_el(&ct.s_full[i]);
        };
        uint32_t c0 = 0;           // tiles of the pieces before
        uint32_t done[2] = {0, 0}; // key tiles of each row tile before
        for (int k = 0; ok && k < kPieces; ++k) {
            Work w;
            if (!piece(k, w)) break;
            const int n_of[2] = {w.n_of[0], w.n_of[1]}, n = max(n_of[0], n_of[1]), j0 = w.j0, keys = w.keys, turn = w.turn;
            ok = n == 0 || full(c0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // (the queries of a tile are there when its results of the piece before have been read)
                ok = ok && wait(&ct.q_full[i][k & 1], (k / 2) & 1);
                if (!ok) break;
                sm100::tc_fence_after();
                if (n_of[i] > 0) scores(i, c0);
            }
            // (only now: a softmax warpgroup without keys here may be a piece ahead, but not two)
            read(k);
            if (ok && n > 0) sm100::mma_commit_el(&ct.empty[c0 % NST]);
            for (int j = 0; j < n && ok; ++j) {
                const bool more = j + 1 < n;
                const uint32_t ck = c0 + 2 * j + 1, cv = c0 + (more ? 2 * j + 2 : 2 * j + 1);
                if (more) ok = full(ck);
                ok = ok && full(cv);
                if (!ok) break;
                const uint32_t v_at = ring_at + (cv % NST) * L::kTileBytes;
                const int at = j + turn < n ? j + turn : j + turn - n;
                const int32_t left = keys - (j0 + at) * kAttnKeys;   // keys from this tile on
                if (left < kAttnKeys) {
                    // value rows behind the last key hold anything
                    uint8_t *v = ring + (cv % NST) * L::kTileBytes;
                    for (int x = lane; x < (kAttnKeys - left) * (D / 8); x += 32)
                        *reinterpret_cast<uint4 *>(v + (x % (D / 8)) / 8 * L::kBlockBytes + (left + x / (D / 8)) * 128 +
                                                   (x % 8) * 16) = make_uint4(0, 0, 0, 0);
                    sm100::fence_proxy_async_smem();
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (j < n_of[i]) {
                        ok = wait(&ct.p_ready[i], (done[i] + j) & 1);
                        if (!ok) break;
                        sm100::tc_fence_after();
#pragma unroll
                        for (int s = 0; s < kAttnKeys / 16; ++s)
                            mma16_ts(tmem + 256 + i * D, tmem + i * 128 + s * 8, sdesc_mn(v_at + s * 2048, L::kBlockBytes),
                                     idesc_16(BF16, 128, D, true), j > 0 || s > 0);
                        if (j == n_of[i] - 1) sm100::mma_commit_el(&ct.o_full[i]);
                    }
                    if (j + 1 < n_of[i]) scores(i, ck);
                }
                if (!ok) break;
                sm100::mma_commit_el(&ct.empty[cv % NST]);
                if (more) sm100::mma_commit_el(&ct.empty[ck % NST]);
            }
            c0 += 2 * n;
            done[0] += n_of[0];
            done[1] += n_of[1];
        }
        // whatever was issued is over before the block ends
        sm100::mma_commit_el(&ct.done);
        attn_wait(&ct.done, 0, &g_attn_status);
    } else if (warp < 8) {
        // ------------------------------------------------ softmax: one thread a row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int i = warp >> 2, rt = tid & 127;             // row tile, row of it
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t S = lanes + i * 128, O = lanes + 256 + i * D;
        const float c = A.scale_log2;
        const uint64_t c2 = pack2(c, c);
        uint32_t done = 0, outs = 0;   // key tiles, and pieces with any, before
        for (int k = 0; ok && k < kPieces; ++k) {
            Work w;
            if (!piece(k, w)) break;
            const int32_t tile = w.tile, head = w.head, rows = w.rows, j0 = w.j0, mine = i ? w.n_of[1] : w.n_of[0], slot = w.slot, keys = w.keys;
            const int32_t n = max(w.n_of[0], w.n_of[1]), turn = w.turn;
            const int32_t behind = keys - w.tokens;   // key index that the first token sees last
            const int64_t a = w.a;
            read(k);
            if (k > 0) sm100::named_sync(1 + i, 128);   // the tile's results have left its place
            {
                // 16 bytes a thread and pass, all passes in flight; a short loop, because code that runs once a
                // block is paid by its length
                constexpr int CH = D / 8, PER = 128 / CH;   // 16-byte pieces of a row; rows a pass
                const int p = rt % CH;
                int r = rt / CH;
                Row at(tile * kTileRows + i * 128 + r, G);
                const Row step(PER, G);
                const uint16_t *q = static_cast<const uint16_t *>(A.q) + a * A.q_t + (int64_t)head * G * A.q_h + p * 8;
                uint32_t to = sm100::smem_u32(Qs + i * L::kTileBytes + (p >> 3) * L::kBlockBytes + ((p & 7) << 4));
#pragma unroll 4
                for (int x = 0; x < CH; ++x, r += PER) {
                    const bool some = i * 128 + r < rows;   // else zeros
                    cp_async16(to + r * 128 ^ ((r & 7) << 4), some ? q + at.tok * A.q_t + at.g * A.q_h : q, some ? 16 : 0);
                    at.add(step, G);
                }
                sm100::cp_async_wait_all();
                sm100::fence_proxy_async_smem();
                sm100::mbar_arrive(&ct.q_full[i][k & 1]);
            }
            const int r = i * 128 + rt, fr = tile * kTileRows + r, tok = fr / G, g = fr - tok * G;
            const bool live = r < rows;
            const int32_t seen = live ? max(0, min(behind + tok + 1, keys)) : 0;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < mine; ++j) {
                ok = attn_wait(&ct.s_full[i], (done + j) & 1, &g_attn_status);
                if (!ok) break;
                sm100::tc_fence_after();
                float s[128];
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_ld32_nowait(S + x * 32, s + x * 32);
                tmem_wait_ld(s);
                const int32_t vis = seen - (j0 + (j + turn < n ? j + turn : j + turn - n)) * kAttnKeys;
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
                const bool grown = top > m && (top - m) * c > kGrowth<BF16>;   // also from -inf
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
                const float shift = m == -INFINITY ? 0.f : kUp<BF16> - m * c;
                const uint64_t s2 = pack2(shift, shift);
                uint64_t sum[2] = {0, 0};
                uint32_t p[64];
#pragma unroll
                for (int x = 0; x < 64; ++x) {
                    float y, z;
                    unpack2(fma2(pack2(s[2 * x], s[2 * x + 1]), c2, s2), y, z);
                    y = ex2(y);
                    z = ex2(z);
                    sum[x & 1] = add2(sum[x & 1], pack2(y, z));
                    p[x] = pack16<BF16>(y, z);
                    if ((x & 15) == 15) tmem_st16_raw(S + (x & ~15), p + (x & ~15));
                }
                float y, z;
                unpack2(add2(sum[0], sum[1]), y, z);
                l += y + z;
                sm100::tmem_wait_st();
                sm100::tc_fence_before();
                sm100::mbar_arrive(&ct.p_ready[i]);
            }
            done += mine;
            if (mine > 0) {
                ok = ok && attn_wait(&ct.o_full[i], outs++ & 1, &g_attn_status);
                sm100::tc_fence_after();
            }
            if (!ok) break;
            // ------------------------------------------------ results
            // A row whose sum is 0 has seen no key (or scores of -inf only): out 0.  A sum that is
            // NaN reaches the row through 1 / l.
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            const float lse = l > 0.f || l != l ? m * A.scale + logf(plain_sum<BF16>(l)) : -INFINITY;
            const bool share = PAGED && slot >= 0;
            const int64_t at = a + tok;
            const int h = head * G + g;
            // Through the tile's queries in shared memory (their products are over), so that a warp
            // writes whole rows.
            uint8_t *stage = Qs + i * L::kTileBytes + (rt & ~31) * (D * 2);
            const bool f32 = share || A.out_dtype == KDA_DTYPE_F32;
            const int rounds = f32 ? 2 : 1, width = f32 ? D / 2 : D;   // D * 2 bytes of a row a round
#pragma unroll 1
            for (int round = 0; round < rounds; ++round) {
#pragma unroll 1
                for (int x = 0; x < width; x += 32) {
                    float o[32];
                    if (mine > 0) {
                        tmem_ld32_nowait(O + round * width + x, o);
                        tmem_wait_ld(o);
                    }
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = inv == 0.f ? 0.f : o[y] * inv;
                    // piece x / 8 (16-bit) or x / 4 (fp32) of the row, turned within eight
                    uint8_t *row = stage + lane * (D * 2);
                    if (f32) {
#pragma unroll
                        for (int y = 0; y < 32; y += 4)
                            *reinterpret_cast<float4 *>(row + ((((x + y) >> 2) ^ (lane & 7)) << 4)) =
                                make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; y += 8)
                            *reinterpret_cast<uint4 *>(row + ((((x + y) >> 3) ^ (lane & 7)) << 4)) =
                                make_uint4(pack16<BF16>(o[y], o[y + 1]), pack16<BF16>(o[y + 2], o[y + 3]),
                                           pack16<BF16>(o[y + 4], o[y + 5]), pack16<BF16>(o[y + 6], o[y + 7]));
                    }
                }
                __syncwarp();
                constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;   // lanes a row, rows a pass
                const int p = lane % LANES;
                int rr = lane / LANES, br = i * 128 + (rt & ~31) + rr;   // row of the warp, of the block
                Row here(tile * kTileRows + br, G);
                const Row step(AT_ONCE, G);
                uint8_t *to = static_cast<uint8_t *>(share ? (void *)sh.out : A.out) + round * (D * 2) + p * 16;
#pragma unroll 1
                for (; rr < 32 && br < rows; rr += AT_ONCE, br += AT_ONCE) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(stage + rr * (D * 2) + ((p ^ (rr & 7)) << 4));
                    const int64_t row = share ? (int64_t)slot * kTileRows + br : (a + here.tok) * A.Hq + head * G + here.g;
                    *reinterpret_cast<uint4 *>(to + row * rounds * (D * 2)) = v;
                    here.add(step, G);
                }
                __syncwarp();
            }
            if (live) {
                if (share)
                    sh.lse[(int64_t)slot * kTileRows + r] = lse;
                else if (A.lse)
                    A.lse[at * A.Hq + h] = lse;
            }
            sm100::tc_fence_before();
        }
        sm100::tc_fence_before();
    }
    __syncthreads();
    if (warp == kProductWarp) sm100::tmem_dealloc(tmem, 512);
}

// Joins the shares of a split row tile: out = sum_s w_s out_s with w_s = e^(lse_s - lse), in the
// order of the shares.  One warp has a row, or the four of a block together where there are many
// shares (a lane has D / 32 channels; all loads of a warp are in flight at once).
template <int D, bool BF16>
__device__ __forceinline__ void join_row(const Attn &A, const float *lse, const float *out, int rows, int second, int step,
                                         int splits, int64_t at, bool together, float (*part)[D + 2]) {
    // the first share's row is at lse and out; the others' slots (of `rows` rows) follow
    auto off = [&](int s) { return s ? (int64_t)(second + (s - 1) * step) * rows : 0; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = together ? warp : 0, stride = together ? 4 : 1;
    constexpr int PER = D / 32;
    float top = -INFINITY;
    for (int s = lane; s < splits; s += 32) top = fmaxf(top, lse[off(s)]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc[PER] = {};
    for (int s0 = first; s0 < splits; s0 += stride * 8) {
        float w[8], v[8][PER];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int s = s0 + x * stride;
            w[x] = s < splits ? lse[off(s)] : -INFINITY;
#pragma unroll
            for (int y = 0; y < PER; y += 2) {
                const float2 z = s < splits ? *reinterpret_cast<const float2 *>(out + off(s) * D + lane * PER + y)
                                            : make_float2(0.f, 0.f);
                v[x][y] = z.x;
                v[x][y + 1] = z.y;
            }
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            w[x] = __expf(w[x] - ref);
            sum += w[x];
#pragma unroll
            for (int y = 0; y < PER; ++y) acc[y] += w[x] == 0.f ? 0.f : w[x] * v[x][y];
        }
    }
    if (together) {
        if (lane == 0) part[warp][D] = sum;
#pragma unroll
        for (int y = 0; y < PER; ++y) part[warp][lane * PER + y] = acc[y];
        __syncthreads();
        sum = (part[0][D] + part[1][D]) + (part[2][D] + part[3][D]);
#pragma unroll
        for (int y = 0; y < PER; ++y) {
            const int ch = lane * PER + y;
            acc[y] = (part[0][ch] + part[1][ch]) + (part[2][ch] + part[3][ch]);
        }
        __syncthreads();
        if (warp != 0) return;
    }
    const bool none = !(sum > 0.f) && sum == sum;   // no key seen anywhere
    const float inv = none ? 0.f : 1.f / sum;
#pragma unroll
    for (int y = 0; y < PER; y += 2) {
        if (A.out_dtype == KDA_DTYPE_F32)
            *reinterpret_cast<float2 *>(static_cast<float *>(A.out) + at * D + lane * PER + y) =
                make_float2(acc[y] * inv, acc[y + 1] * inv);
        else
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(A.out) + at * D + lane * PER + y) =
                pack16<BF16>(acc[y] * inv, acc[y + 1] * inv);
    }
    if (lane == 0 && A.lse) A.lse[at] = none ? -INFINITY : top + logf(sum);
}

// Shares of kda_attn_tc_kernel: the block that began a row tile left a record; its share is the
// second of that block's two slots, the others are the first of the next blocks'.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) kda_attn_join_kernel(const Attn A, const Shares sh) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x;
    const int32_t splits = sh.rec[b * 4];
    if (splits == 0) return;
    const int n = sh.rec[b * 4 + 1], tile = sh.rec[b * 4 + 2], head = sh.rec[b * 4 + 3];
    int64_t a, e;
    seq_bounds(A.cu, n, A.T, A.seq_len, a, e);
    const int64_t rows = (e - a) * A.G - (int64_t)tile * kTileRows;
    for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < kTileRows && r < rows; r += gridDim.y * 4) {
        const int64_t fr = (int64_t)tile * kTileRows + r, tok = fr / A.G;
        const int64_t slot = 2 * (int64_t)b + 1;
        join_row<D, BF16>(A, sh.lse + slot * kTileRows + r, sh.out + (slot * kTileRows + r) * D, kTileRows, 1, 2, splits,
                          (a + tok) * A.Hq + head * A.G + (fr - tok * A.G), false, nullptr);
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
        sm100::prefetch_tmap(&kmap);
        sm100::prefetch_tmap(&vmap);
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
    AttnPart part;
    if (!attn_split_part<kFewThreads>(A.N, A.Hkv, blockIdx.x, slots_at_once, 8, 4, need, part, &ct.part, ct.scan)) return;
    const AttnSeq sq = attn_seq<true>(A, part.n);
    if (part.split == 0 && tid == 0) {
        int32_t *rec = sh.rec + ((int64_t)part.n * A.Hkv + part.head) * 4;
        rec[0] = part.splits;
        rec[1] = part.slot;
    }
    const int32_t tokens = (int32_t)(sq.b - sq.a), rows = tokens * G;
    const int32_t behind = (int32_t)sq.keys - tokens, keys = (int32_t)sq.keys;
    const int n = part.j1 - part.j0;
    bool ok = true;
    if (warp == 4) {
        const int boxes = kFewKeys / box;
        const int unit = lane % (boxes * (D / 64)), mine = unit / boxes, which = unit % boxes;
        const bool values = lane >= boxes * (D / 64), issues = lane < 2 * boxes * (D / 64);
        const int32_t *row = A.table + (int64_t)part.n * A.wide;
        bool bad = A.lens[part.n] > (int64_t)A.wide * A.page;
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
        const bool g0 = t0 > m0 && (t0 - m0) * c > kGrowth<BF16>, g1 = t1 > m1 && (t1 - m1) * c > kGrowth<BF16>;
        if (__any_sync(0xffffffffu, g0 || g1)) {
            const float f0 = g0 ? ex2((m0 - t0) * c) : 1.f, f1 = g1 ? ex2((m1 - t1) * c) : 1.f;
            l0 *= f0;
            l1 *= f1;
            if (g0) m0 = t0;
            if (g1) m1 = t1;
#pragma unroll
            for (int x = 0; x < D / 8; ++x) o[x][0] *= f0, o[x][1] *= f0, o[x][2] *= f1, o[x][3] *= f1;
        }
        const float h0 = m0 == -INFINITY ? 0.f : kUp<BF16> - m0 * c, h1 = m1 == -INFINITY ? 0.f : kUp<BF16> - m1 * c;
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
        // what the 16 bits leave of a weight is a second operand: the products have time for it here, and the
        // result then is as good as fp32 weights would make it
        uint32_t rest[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            float lo, hi;
            unpack16<BF16>(pa[x], lo, hi);
            rest[x] = pack16<BF16>(s[x >> 1][(x & 1) * 2] - lo, s[x >> 1][(x & 1) * 2 + 1] - hi);
        }
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            uint32_t b[4];
            const int piece = x * 2 + vpiece;
            ldsm4_t(b, vb + (piece >> 3) * L::kBlock + vrow * 128 + (((piece & 7) ^ (vrow & 7)) << 4));
            mma16816<BF16>(o[2 * x], pa, b[0], b[1]);
            mma16816<BF16>(o[2 * x + 1], pa, b[2], b[3]);
            mma16816<BF16>(o[2 * x], rest, b[0], b[1]);
            mma16816<BF16>(o[2 * x + 1], rest, b[2], b[3]);
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
        const float lse = none ? -INFINITY : top * A.scale + logf(plain_sum<BF16>(l));
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
}

// Joins the shares of kda_attn_few_kernel: a block has the rows of one sequence and key head,
// every gridDim.y-th of them.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) kda_attn_few_join_kernel(const Attn A, const Shares sh) {
    __shared__ float part[4][D + 2];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = blockIdx.x / A.Hkv, head = blockIdx.x - n * A.Hkv;
    int64_t a, b;
    seq_bounds(A.cu, n, A.T, A.seq_len, a, b);
    const int64_t rows = (b - a) * A.G;
    if (rows == 0 || rows > kFewRows) return;
    const int32_t splits = sh.rec[(int64_t)blockIdx.x * 4], slot = sh.rec[(int64_t)blockIdx.x * 4 + 1];
    if (splits <= 1) return;
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        const int tok = r / A.G;
        join_row<D, BF16>(A, sh.lse + (int64_t)slot * kFewRows + r, sh.out + ((int64_t)slot * kFewRows + r) * D, kFewRows, 1, 1,
                          splits, (a + tok) * A.Hq + head * A.G + (r - tok * A.G), true, part);
    }
}

// ---------------------------------------------------------------- host
// Sizes of a paged call's launches.  Which sequences have few rows is known on the device
// only (unless all are alike): each kernel passes by those that are the other's.
struct Sizes {
    bool many, few;               // launch the kernel of many rows, of few rows
    int64_t few_tiles, few_parts, few_slots;
};
constexpr int kFewAtOnce = 304;   // two blocks an SM

Sizes sizes_of(const Attn &A) {
    Sizes z{};
    if (A.N == 0 || A.T == 0) return z;
    z.few = A.cu ? true : A.seq_len * A.G <= kFewRows;
    z.many = A.cu ? (int64_t)A.T * A.G > kFewRows : !z.few;
    if (z.few) {
        z.few_tiles = (int64_t)A.N * A.Hkv;
        z.few_parts = attn_parts(z.few_tiles, kFewAtOnce, 8);
        // a sequence that is cut has more than one run of keys: at most two parts a run
        z.few_slots = z.few_parts < 16 * kFewAtOnce ? z.few_parts : 16 * kFewAtOnce;
    }
    return z;
}

int64_t up(int64_t x) { return (x + 255) / 256 * 256; }
int64_t shares_bytes(int64_t records, int64_t slots, int rows, int d) {
    return up(records * 16) + up(slots * rows * 4) + up(slots * rows * d * 4);
}

Shares shares_at(char *ws, int64_t records, int64_t slots, int rows) {
    Shares s;
    s.rec = reinterpret_cast<int32_t *>(ws);
    s.lse = reinterpret_cast<float *>(ws + up(records * 16));
    s.out = reinterpret_cast<float *>(ws + up(records * 16) + up(slots * rows * 4));
    return s;
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
    cudaError_t e = kda_allow_smem<kda_attn_tc_kernel<D, BF16, false>>(Lay<D>::kSmem);
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
        const Shares sh = shares_at(ws, z.few_tiles, z.few_slots, kFewRows);
        const auto kernel = kda_attn_few_kernel<D, BF16>;
        e = kda_allow_smem<kda_attn_few_kernel<D, BF16>>(FewLay<D>::kSmem);
        if (e == cudaSuccess)
            e = launch(false, kernel, dim3((unsigned)z.few_parts), kFewThreads, FewLay<D>::kSmem, stream, km, vm, A, sh,
                       box, kFewAtOnce);
        if (e == cudaSuccess)
            e = launch(true, kda_attn_few_join_kernel<D, BF16>,
                       dim3((unsigned)z.few_tiles, (unsigned)(z.few_tiles < kFewAtOnce ? (A.G < kFewRows ? A.G : kFewRows) : 1)),
                       128, 0, stream, A, sh);
        ws += shares_bytes(z.few_tiles, z.few_slots, kFewRows, D);
    }
    if (z.many && e == cudaSuccess) {
        const int box = A.page < kAttnKeys ? A.page : kAttnKeys;
        CUtensorMap km, vm;
        if (!kda_make_attn_map(&km, A.k, BF16, D, A.Hkv, A.page, A.P, A.k_h, A.k_t, A.k_p, box) ||
            !kda_make_attn_map(&vm, A.v, BF16, D, A.Hkv, A.page, A.P, A.v_h, A.v_t, A.v_p, box))
            return cudaErrorInvalidValue;
        const Shares sh = shares_at(ws, kSMs, 2 * kSMs, kTileRows);
        const auto kernel = kda_attn_tc_kernel<D, BF16, true>;
        e = kda_allow_smem<kda_attn_tc_kernel<D, BF16, true>>(Lay<D>::kSmem);
        if (e == cudaSuccess)
            e = launch(false, kernel, dim3(kSMs), kThreads, Lay<D>::kSmem, stream, km, vm, A, sh, box,
                       z.few ? kFewRows : 0);
        if (e == cudaSuccess)
            e = launch(true, kda_attn_join_kernel<D, BF16>, dim3(kSMs, 32), 128, 0, stream, A, sh);
    }
    return e;
}

}  // namespace

int64_t kda_attn_paged_ws(const Attn &A) {
    const Sizes z = sizes_of(A);
    return (z.few ? shares_bytes(z.few_tiles, z.few_slots, kFewRows, A.d) : 0) +
           (z.many ? shares_bytes(kSMs, 2 * kSMs, kTileRows, A.d) : 0);
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
