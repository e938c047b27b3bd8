// kda_attn_plan.cuh -- which part of a packed batch a block works on.  The lengths are
// known on the device only, so every block finds its own part: each thread counts the
// parts of a run of sequences, and one scan over the block says whose run holds the
// block's number.  A batch of 256 sequences costs a block about a microsecond.
#pragma once

#include "kda_attn_common.cuh"

namespace kda {

// One block's part of the work: query rows [tile * rows of a tile, ...) of sequence n
// against key tiles [j0, j1); `slot`: where a share of a split row tile goes (-1: the part
// is all of it).
struct AttnPart {
    int32_t n, tile, head, j0, j1, split, splits, slot;
};

// Exclusive sums over the block's threads; `total` of all.  Every thread calls it.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t &total, int64_t *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = s;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sh[w];
        all += sh[w];
    }
    total = all;
    return before + s - x;
}

// What a sequence needs: its row tiles and the key tiles of each (0 row tiles: none here).
struct AttnNeed {
    int32_t tiles, keys;
};

// Longest key run of a part, by the number of row tiles (times heads) and their key tiles.
// Few row tiles: as many parts as `slots` blocks run at once, so that all run side by
// side.  More: runs short enough that the last ones to finish do not matter.  Enough:
// row tiles are not cut.
__host__ __device__ inline int32_t attn_run(int64_t tiles, int64_t keys, int slots, int waves, int least) {
    if (tiles >= (int64_t)slots * waves) return INT32_MAX;
    const int64_t parts = tiles * 2 <= slots ? slots - tiles : (int64_t)slots * waves;
    int64_t run = (keys + parts - 1) / parts;
    if (run < least) run = least;
    return run > INT32_MAX ? INT32_MAX : (int32_t)run;
}
// Upper bounds on the parts, and on those of them that are shares, of `tiles` row tiles at most.
__host__ inline int64_t attn_parts(int64_t tiles, int slots, int waves) {
    return tiles * 2 <= slots ? slots : tiles + (int64_t)slots * waves;
}

// Part number `index` of `heads` heads (head fastest).  `need(n)` gives what sequence n needs.  False:
// there is no such part.  Up to 32 sequences each warp finds it by itself (and the block only
// meets); beyond, the block does together.  Every thread calls it.
template <int THREADS, typename Need>
__device__ __forceinline__ bool attn_split_part(int N, int heads, int64_t index, int slots, int waves, int least,
                                                Need need, AttnPart &part, AttnPart *shared, int64_t *sh) {
    const int64_t at = index / heads;
    auto fill = [&](AttnPart &p, int n, const AttnNeed &x, int32_t run, int64_t splits, int64_t in, int64_t shares_before) {
        p.n = n;
        p.head = (int32_t)(index - at * heads);
        p.tile = (int32_t)(in / splits);
        p.split = (int32_t)(in - p.tile * splits);
        p.splits = (int32_t)splits;
        p.j0 = splits > 1 ? p.split * run : 0;
        p.j1 = splits > 1 ? min(x.keys, p.j0 + run) : x.keys;
        p.slot = splits > 1 ? (int32_t)((shares_before + p.tile * splits) * heads + (int64_t)p.head * splits + p.split) : -1;
    };
    auto splits_of = [](const AttnNeed &x, int32_t run) { return x.keys > run ? (int64_t)(x.keys + run - 1) / run : (int64_t)1; };
    if (N <= 32) {
        const int lane = threadIdx.x & 31;
        const AttnNeed x = lane < N ? need(lane) : AttnNeed{0, 0};
        int64_t tiles = x.tiles, keys = (int64_t)x.tiles * x.keys;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
            keys += __shfl_xor_sync(0xffffffffu, keys, o);
        }
        const int32_t run = attn_run(tiles * heads, keys * heads, slots, waves, least);
        const int64_t splits = splits_of(x, run), parts = x.tiles * splits, shares = splits > 1 ? parts : 0;
        int64_t p = parts, s = shares;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, p, o), z = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) p += y, s += z;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, at >= p - parts && at < p);
        __syncthreads();
        if (!here) return false;
        const int n = __ffs(here) - 1;
        const AttnNeed y{__shfl_sync(0xffffffffu, x.tiles, n), __shfl_sync(0xffffffffu, x.keys, n)};
        fill(part, n, y, run, __shfl_sync(0xffffffffu, splits, n), at - __shfl_sync(0xffffffffu, p - parts, n),
             __shfl_sync(0xffffffffu, s - shares, n));
        return true;
    }
    const int per = (N + THREADS - 1) / THREADS;
    const int lo = (int)threadIdx.x * per, hi = min(N, lo + per);
    int64_t tiles = 0, keys = 0, total_tiles, total_keys;
    for (int n = lo; n < hi; ++n) {
        const AttnNeed x = need(n);
        tiles += x.tiles;
        keys += (int64_t)x.tiles * x.keys;
    }
    block_scan<THREADS>(tiles, total_tiles, sh);
    block_scan<THREADS>(keys, total_keys, sh);
    const int32_t run = attn_run(total_tiles * heads, total_keys * heads, slots, waves, least);
    int64_t parts = 0, shares = 0, total_parts, total_shares;
    for (int n = lo; n < hi; ++n) {
        const AttnNeed x = need(n);
        const int64_t splits = splits_of(x, run);
        parts += x.tiles * splits;
        if (splits > 1) shares += x.tiles * splits;
    }
    int64_t before = block_scan<THREADS>(parts, total_parts, sh);
    int64_t shares_before = block_scan<THREADS>(shares, total_shares, sh);
    if (at >= total_parts) return false;
    if (at >= before && at < before + parts) {
        for (int n = lo; n < hi; ++n) {
            const AttnNeed x = need(n);
            const int64_t splits = splits_of(x, run);
            if (at < before + x.tiles * splits) {
                fill(*shared, n, x, run, splits, at - before, shares_before);
                break;
            }
            before += x.tiles * splits;
            if (splits > 1) shares_before += x.tiles * splits;
        }
    }
    __syncthreads();
    part = *shared;
    return true;
}

// A warp's inclusive sums.
__device__ __forceinline__ int64_t warp_scan(int64_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Of up to 32 sequences, the one that holds unit `at`, by a warp: lane n has the `units` of sequence n.
// `first`: its first unit; -1: none holds it.
__device__ __forceinline__ int warp_find(int64_t units, int64_t at, int64_t &first) {
    const int64_t upto = warp_scan(units);
    const uint32_t here = __ballot_sync(0xffffffffu, at >= upto - units && at < upto);
    const int n = __ffs(here) - 1;
    first = __shfl_sync(0xffffffffu, upto - units, n < 0 ? 0 : n);
    return n;
}

// Tile number `index` of `heads` heads (head fastest), from the first tile to the last or, with
// `reverse`, from the last to the first: what takes longest starts first.  `same` >= 0: every
// sequence has that many tiles.  Then, and up to 32 sequences, each warp finds it by itself;
// beyond, the block does together.  Every thread calls it.
template <int THREADS, typename Tiles>
__device__ __forceinline__ bool attn_whole_part(int N, int heads, uint32_t index, bool reverse, int same, Tiles tiles_of,
                                                AttnPart &part, AttnPart *shared, int64_t *sh) {
    const uint32_t head = index % (uint32_t)heads, tile = index / (uint32_t)heads;
    part.head = (int32_t)head;
    part.slot = -1;
    part.splits = 1;
    if (same >= 0) {
        const uint32_t total = (uint32_t)N * (uint32_t)same;   // (fits: the grid holds that many blocks)
        if (tile >= total) return false;
        const uint32_t at = reverse ? total - 1 - tile : tile;
        part.n = (int32_t)(at / (uint32_t)same);
        part.tile = (int32_t)(at % (uint32_t)same);
        return true;
    }
    if (N <= 32) {
        const int lane = threadIdx.x & 31;
        const int64_t tiles = lane < N ? tiles_of(lane) : 0, total = __shfl_sync(0xffffffffu, warp_scan(tiles), 31);
        if (tile >= total) return false;
        int64_t first;
        const int64_t at = reverse ? total - 1 - tile : tile;
        part.n = warp_find(tiles, at, first);
        part.tile = (int32_t)(at - first);
        return true;
    }
    const int per = (N + THREADS - 1) / THREADS;
    const int lo = (int)threadIdx.x * per, hi = min(N, lo + per);
    int64_t tiles = 0, total;
    for (int n = lo; n < hi; ++n) tiles += tiles_of(n);
    int64_t before = block_scan<THREADS>(tiles, total, sh);
    if (tile >= total) return false;
    const int64_t at = reverse ? total - 1 - tile : tile;
    if (at >= before && at < before + tiles) {
        for (int n = lo; n < hi; ++n) {
            const int64_t x = tiles_of(n);
            if (at < before + x) {
                shared->n = n;
                shared->tile = (int32_t)(at - before);
                break;
            }
            before += x;
        }
    }
    __syncthreads();
    part.n = shared->n;
    part.tile = shared->tile;
    return true;
}

}  // namespace kda
