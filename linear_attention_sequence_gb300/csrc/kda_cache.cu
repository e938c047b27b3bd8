// kda_cache.cu -- the pages of a cache of keys and values: taking pages for new tokens,
// writing the tokens, sharing pages between continuations of a prompt, giving pages
// back, and moving the pages in use together.  Everything that decides which page goes
// where is done on the device, so that a decode loop of captured graphs never waits for
// the host; and everything is decided by number order (lowest free page first, sequences in
// their order), so that the same calls give the same tables every time.
//
// Two kinds of kernels: bookkeeping on counts and tables (a few hundred KB at most: latency
// bounds it, so that each call is one or two launches), and copies of keys and values (HBM
// bounds them; 16-byte accesses, several in flight a thread).
#include <cooperative_groups.h>

#include "kda_cache.cuh"

namespace cg = cooperative_groups;
using namespace kda;

namespace {

__device__ unsigned g_cache_status;

constexpr int kBlock = 1024;

__device__ __forceinline__ int pages_of(int64_t tokens, int shift) {
    return (int)((tokens + (1 << shift) - 1) >> shift);
}
// A sequence's length, within what its table row can hold.
__device__ __forceinline__ int length_of(const Cache &C, int n) {
    const int len = C.lens[n];
    return len < 0 ? 0 : min(len, C.wide << C.shift);
}

// Exclusive sum over the 1024 threads, and the total (of one count, or of two in the halves of 64
// bits).
template <typename T>
__device__ __forceinline__ T scan1024(T x, T &total, T *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = s;
    __syncthreads();
    T w = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const T before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp ? before : 0) + s - x;
}
typedef unsigned long long Two;   // a count in the low half, another in the high half
__device__ __forceinline__ Two two(int a, int b) { return (Two)(unsigned)a | (Two)(unsigned)b << 32; }

// The first `want` free pages, lowest first, into `list`; returns how many there are (no
// more than `want`).  The counts are read 16 a thread and step, the next step's ahead.
__device__ int free_pages(const int32_t *refs, int P, int want, int32_t *list, int *sh) {
    constexpr int PER = 16;
    int found = 0;
    for (int base = 0; base < P && found < want; base += kBlock * PER) {
        const int first = base + (int)threadIdx.x * PER;
        uint32_t free = 0;
        if (first + PER <= P && ((uintptr_t)refs & 15) == 0) {
            const int4 *p = reinterpret_cast<const int4 *>(refs + first);
            int4 v[PER / 4];
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) v[i] = p[i];
#pragma unroll
            for (int i = 0; i < PER / 4; ++i)
                free |= ((v[i].x == 0) | (v[i].y == 0) << 1 | (v[i].z == 0) << 2 | (v[i].w == 0) << 3) << (4 * i);
        } else {
            for (int i = 0; i < PER; ++i)
                if (first + i < P && refs[first + i] == 0) free |= 1u << i;
        }
        int total;
        int at = found + scan1024(__popc(free), total, sh);
        while (free && at < want) {
            list[at++] = first + __ffs(free) - 1;
            free &= free - 1;
        }
        found += total;
    }
    __syncthreads();   // the list is read by all threads
    return min(found, want);
}

// ---------------------------------------------------------------- reserve
// A last page that is not full and that others share (a sequence was shortened into it) is replaced
// by one of the sequence's own.  Which sequences that is, is settled before any count changes (src).
__global__ void __launch_bounds__(kBlock) kda_cache_reserve_kernel(const Cache C, const int32_t *new_lens, int32_t *src,
                                                                   int32_t *dst, int32_t *missing, int32_t *granted, int32_t *list) {
    __shared__ int sh[32];
    auto shared_page = [&](int n, int len, int add) {
        if (add == 0 || (len & ((1 << C.shift) - 1)) == 0) return -1;
        const int p = C.table[(int64_t)n * C.wide + (len >> C.shift)];
        return p >= 0 && p < C.P && C.refs[p] > 1 ? p : -1;
    };
    // (new pages; -1: the table's row is too short, or a page to copy and nowhere to say so)
    auto needs = [&](int n, bool first, int &len, int &add, int &have, int &old) {
        len = length_of(C, n);
        add = max(0, new_lens[n]);
        have = pages_of(len, C.shift);
        old = src && !first ? src[n] : shared_page(n, len, add);
        const int64_t want = ((int64_t)len + add + (1 << C.shift) - 1) >> C.shift;
        if (first && src) src[n] = old;
        if (old >= 0 && !src) {
            if (first) atomicOr(&g_cache_status, kCacheBadPage);
            return -1;
        }
        return want > C.wide ? -1 : (int)want - have + (old >= 0);
    };
    // how many pages in all
    int64_t want = 0;
    for (int base = 0; base < C.N; base += kBlock) {
        const int n = base + threadIdx.x;
        int len, add, have, old, total;
        const int need = n < C.N ? max(0, needs(n, true, len, add, have, old)) : 0;
        scan1024(need, total, sh);   // (N * wide fits 32 bits)
        want += total;
    }
    const int ask = (int)min(want, (int64_t)C.P);
    const int got = ask ? free_pages(C.refs, C.P, ask, list, sh) : 0;
    if (missing && threadIdx.x == 0) *missing = (int)min(want - got, (int64_t)INT32_MAX);
    int64_t before = 0;
    for (int base = 0; base < C.N; base += kBlock) {
        const int n = base + threadIdx.x;
        int len = 0, add = 0, have = 0, old = -1, total;
        const int need = n < C.N ? needs(n, false, len, add, have, old) : -1;
        const int64_t at = before + scan1024(max(0, need), total, sh);
        before += total;
        if (n >= C.N) continue;
        const bool served = need >= 0 && (need == 0 || at + need <= got);
        const int copies = served && old >= 0 ? 1 : 0;
        if (src) {
            src[n] = copies ? old : -1;
            dst[n] = copies ? list[at] : -1;
        }
        // a refusal is told to whoever appends next, or recorded
        if (granted)
            granted[n] = served ? add : 0;
        else if (!served && !missing)
            atomicOr(&g_cache_status, kCacheBadPage);
        if (!served) continue;
        int32_t *row = C.table + (int64_t)n * C.wide + have - copies;
        if (copies) atomicSub(C.refs + old, 1);
        for (int j = 0; j < need; ++j) {
            const int p = list[at + j];
            row[j] = p;
            C.refs[p] = 1;
        }
        C.lens[n] = len + add;
    }
}

// ---------------------------------------------------------------- append
// Rows are written 16 bytes a thread; a block of 256 threads takes kAppendTokens tokens and
// first finds where each goes.
constexpr int kAppendTokens = 8;
__global__ void __launch_bounds__(256) kda_cache_append_kernel(const Cache C, const Heads k, const Heads v, const Pages kp,
                                                               const Pages vp, const int32_t *cu, int64_t T, int64_t seq_len,
                                                               const int32_t *granted) {
    __shared__ int64_t to_k[kAppendTokens], to_v[kAppendTokens];
    const int64_t first = (int64_t)blockIdx.x * kAppendTokens;
    if (threadIdx.x < kAppendTokens) {
        const int64_t t = first + threadIdx.x;
        to_k[threadIdx.x] = -1;
        int n = -1;
        int64_t a = 0, b = 0;
        if (t < T && C.N > 0) {
            if (!cu) {
                n = (int)(t / seq_len);
                a = n * seq_len, b = a + seq_len;
            } else {
                // the last sequence that starts at t or before it (empty ones come before it)
                int lo = 0, hi = C.N;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (cu[mid] <= t) lo = mid; else hi = mid;
                }
                seq_bounds(cu, lo, T, 0, a, b);
                if (t >= a && t < b) n = lo;
            }
        }
        // (refused: kv_lens does not count these tokens, and the places in front of it hold others)
        if (n >= 0 && !(granted && granted[n] < b - a)) {
            const int len = C.lens[n];
            const int64_t at = (int64_t)len - (b - a) + (t - a);
            if (len > (int64_t)C.wide << C.shift) {
                atomicOr(&g_cache_status, kCacheBadPage);
            } else if (at >= 0) {
                const int p = C.table[(int64_t)n * C.wide + (at >> C.shift)];
                const int64_t in = at & ((1 << C.shift) - 1);
                if (p < 0 || p >= C.P) {
                    atomicOr(&g_cache_status, kCacheBadPage);
                } else {
                    to_k[threadIdx.x] = p * kp.page + in * kp.token;
                    to_v[threadIdx.x] = p * vp.page + in * vp.token;
                }
            }
        }
    }
    __syncthreads();
    const int pieces = C.d / 8, row = C.H * pieces;   // 16-byte pieces of a token's keys
    for (int x = threadIdx.x; x < kAppendTokens * row; x += 256) {
        const int i = x / row, y = x - i * row, h = y / pieces, c = (y - h * pieces) * 8;
        if (to_k[i] < 0) continue;
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(k.p + (first + i) * k.token + h * k.head + c));
        const uint4 b = __ldg(reinterpret_cast<const uint4 *>(v.p + (first + i) * v.token + h * v.head + c));
        *reinterpret_cast<uint4 *>(kp.p + to_k[i] + h * kp.head + c) = a;
        *reinterpret_cast<uint4 *>(vp.p + to_v[i] + h * vp.head + c) = b;
    }
}

// ---------------------------------------------------------------- free
// A block a listed sequence.  The length is lowered atomically, and whoever lowered it gives
// back the pages between: a sequence that is listed twice gives each page back once.
__global__ void __launch_bounds__(256) kda_cache_free_kernel(const Cache C, const int32_t *seqs, const int32_t *keep) {
    __shared__ int range[2];
    const int n = seqs[blockIdx.x];
    if (n < 0 || n >= C.N) {
        if (threadIdx.x == 0) atomicOr(&g_cache_status, kCacheBadPage);
        return;
    }
    if (threadIdx.x == 0) {
        const int left = keep ? max(0, keep[blockIdx.x]) : 0;
        const int old = min(atomicMin(C.lens + n, left), C.wide << C.shift);
        range[0] = pages_of(left, C.shift);
        range[1] = old > left ? pages_of(old, C.shift) : 0;
    }
    __syncthreads();
    int32_t *row = C.table + (int64_t)n * C.wide;
    for (int j = range[0] + threadIdx.x; j < range[1]; j += 256) {
        const int p = row[j];
        row[j] = -1;
        if (p >= 0 && p < C.P)
            atomicSub(C.refs + p, 1);
        else
            atomicOr(&g_cache_status, kCacheBadPage);
    }
}

// ---------------------------------------------------------------- fork
// First a page for each child whose parent's last page is not full (one block; src and dst
// are the pages to be copied), then the children's rows: a block each in a second kernel, or, where
// they are few entries, a warp each in the first (a launch costs the host as much as the work).
// What a child must be: an empty row (a row with pages would leave their counts behind).  The rows are
// written after the last block has asked for its pages, so that a row's own answer holds throughout.
__device__ __forceinline__ bool may_fork(const Cache &C, int parent, int child) {
    return parent >= 0 && parent < C.N && child >= 0 && child < C.N && parent != child && C.table[(int64_t)child * C.wide] < 0;
}
__device__ __forceinline__ void fork_row(const Cache &C, int parent, int child, int own, int first, int step) {
    const int len = length_of(C, child), whole = len >> C.shift;
    const int32_t *from = C.table + (int64_t)parent * C.wide;
    int32_t *to = C.table + (int64_t)child * C.wide;
    for (int j = first; j < C.wide; j += step) {
        int p = -1;
        if (j < whole) {
            p = from[j];
            if (p >= 0 && p < C.P)
                atomicAdd(C.refs + p, 1);
            else
                atomicOr(&g_cache_status, kCacheBadPage);
        } else if (j == whole) {
            p = own;
        }
        to[j] = p;
    }
}
__global__ void __launch_bounds__(kBlock) kda_cache_fork_pages_kernel(const Cache C, int M, const int32_t *parents,
                                                                      const int32_t *children, int32_t *src, int32_t *dst,
                                                                      int32_t *missing, int32_t *list, bool rows) {
    __shared__ int sh[32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto partial = [&](int m, int &parent, int &child, int &len) {
        parent = parents[m], child = children[m];
        if (!may_fork(C, parent, child)) {
            atomicOr(&g_cache_status, kCacheBadPage);
            return -1;
        }
        len = length_of(C, parent);
        return (len & ((1 << C.shift) - 1)) != 0 ? 1 : 0;
    };
    int want = 0, parent, child, len = 0;
    for (int base = 0; base < M; base += kBlock) {
        const int m = base + threadIdx.x;
        int total;
        scan1024(m < M ? max(0, partial(m, parent, child, len)) : 0, total, sh);
        want += total;
    }
    const int got = want ? free_pages(C.refs, C.P, min(want, C.P), list, sh) : 0;
    if (missing && threadIdx.x == 0) *missing = want - got;
    int before = 0;
    for (int base = 0; base < M; base += kBlock) {
        const int m = base + threadIdx.x;
        int total;
        const int need = m < M ? partial(m, parent, child, len) : -1;
        const int at = before + scan1024(max(0, need), total, sh);
        before += total;
        if (m >= M) continue;
        int from = -1, to = -1;
        if (need >= 0) {
            const bool served = need == 0 || at < got;
            if (need && served) {
                from = C.table[(int64_t)parent * C.wide + (len >> C.shift)];
                to = list[at];
                C.refs[to] = 1;
            }
            C.lens[child] = served ? len : 0;
        }
        src[m] = from;
        dst[m] = to;
    }
    if (!rows) return;
    __syncthreads();
    for (int m = threadIdx.x >> 5; m < M; m += kBlock / 32) {
        parent = parents[m], child = children[m];
        const bool may = may_fork(C, parent, child);
        __syncwarp();   // (asked by all lanes before one writes)
        if (may)
            fork_row(C, parent, child, dst[m], threadIdx.x & 31, 32);
    }
}
__global__ void __launch_bounds__(256) kda_cache_fork_rows_kernel(const Cache C, const int32_t *parents, const int32_t *children,
                                                                  const int32_t *dst) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int parent = parents[blockIdx.x], child = children[blockIdx.x];
    const bool may = may_fork(C, parent, child);
    __syncthreads();    // (asked by all threads before one writes)
    if (!may) return;
    fork_row(C, parent, child, dst[blockIdx.x], threadIdx.x, 256);
}

// ---------------------------------------------------------------- compact
// The pages in use whose numbers are not below their count L move, in order, to the free
// ones that are.  One cluster of eight blocks, each with an eighth of the pages in order, counts and
// lists both sides; then a grid of blocks rewrites the counts and the tables.
constexpr int kCluster = 8;
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kBlock)
    kda_cache_plan_kernel(const int32_t *refs, int P, int32_t *src, int32_t *dst, int32_t *to, int32_t *live_out) {
    __shared__ Two sh[32];
    __shared__ int in_use;
    __shared__ Two counts;   // free below L, in use from L on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int per = ((P + kCluster - 1) / kCluster + 3) & ~3;
    const int lo = min(P, rank * per), hi = min(P, lo + per);
    Two total;
    int mine = 0;
    for (int i = lo + threadIdx.x; i < hi; i += kBlock) mine += refs[i] > 0;
    scan1024(two(mine, 0), total, sh);
    if (threadIdx.x == 0) in_use = (int)total;
    cluster.sync();
    int live = 0;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) live += *cluster.map_shared_rank(&in_use, r);
    Two both = 0;
    for (int i = lo + threadIdx.x; i < hi; i += kBlock) {
        const bool used = refs[i] > 0;
        both += two(!used && i < live, used && i >= live);
    }
    scan1024(both, total, sh);
    if (threadIdx.x == 0) counts = total;
    cluster.sync();
    Two before = 0, all = 0;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) {
        const Two c = *cluster.map_shared_rank(&counts, r);
        if (r < rank) before += c;
        all += c;
    }
    const int moved = (int)all;
    for (int base = lo; base < hi; base += kBlock) {
        const int i = base + threadIdx.x;
        const bool used = i < hi && refs[i] > 0;
        const bool fb = i < hi && !used && i < live, la = used && i >= live;
        const Two at = before + scan1024(two(fb, la), total, sh);
        before += total;
        if (fb) dst[(int)at] = i;
        if (la) src[(int)(at >> 32)] = i;
    }
    // entries behind the moved ones
    for (int i = lo + threadIdx.x; i < hi; i += kBlock)
        if (i >= moved) src[i] = dst[i] = -1;
    cluster.sync();
    for (int i = rank * kBlock + threadIdx.x; i < moved; i += kCluster * kBlock) {
        const int s = *(volatile const int32_t *)(src + i), d = *(volatile const int32_t *)(dst + i);
        to[s] = d;
    }
    if (rank == 0 && threadIdx.x == 0) live_out[0] = live, live_out[1] = moved;
}
__global__ void __launch_bounds__(256) kda_cache_renumber_kernel(const Cache C, const int32_t *src, const int32_t *dst,
                                                                 const int32_t *to, const int32_t *counts, int32_t *refs_out,
                                                                 int32_t *table_out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int live = counts[0], moved = counts[1];
    const int64_t threads = (int64_t)gridDim.x * 256, me = (int64_t)blockIdx.x * 256 + threadIdx.x;
    // counts: a moved page's goes with it; a free page below `live` is written by the one
    // that moves there
    for (int64_t i = me; i < moved; i += threads) {
        const int s = src[i], c = C.refs[s];
        refs_out[dst[i]] = c;
        refs_out[s] = 0;
    }
    if (refs_out != C.refs)
        for (int64_t i = me; i < C.P; i += threads) {
            const int c = C.refs[i];
            if (c > 0 ? i < live : i >= live) refs_out[i] = c;
        }
    const int64_t entries = (int64_t)C.N * C.wide;
    for (int64_t x = me; x < entries; x += threads) {
        const int n = (int)(x / C.wide), j = (int)(x - (int64_t)n * C.wide);
        const int p = C.table[x];
        const bool mine = j < pages_of(length_of(C, n), C.shift);
        int q = p;
        if (mine && p >= live) {
            if (p < C.P)
                q = to[p];
            else
                atomicOr(&g_cache_status, kCacheBadPage);
        }
        if (q != p || table_out != C.table) table_out[x] = q;
    }
}

// ---------------------------------------------------------------- copy
// A unit is a part of one page's keys or values: 16 KB, eight accesses in flight a thread
// (half of a cache of 16384 pages, 0.54 GB: 87 us; with four in flight 101 us, with two 115 us).
// Blocks take units in turn; a lane each looks at the next 32, because a long list may be mostly
// empty entries.
constexpr int kCopyThreads = 128, kCopyInFlight = 8;
template <bool DENSE>
__global__ void __launch_bounds__(kCopyThreads) kda_cache_copy_kernel(const Cache C, const Pages kp, const Pages vp, int M,
                                                                      const int32_t *src, const int32_t *dst) {
    const int pieces = C.d / 8;
    const int page = (C.H * pieces) << C.shift;           // 16-byte pieces of a page
    const int per = (page + kCopyThreads * kCopyInFlight - 1) / (kCopyThreads * kCopyInFlight);
    const int64_t units = (int64_t)M * per * 2;
    const int lane = threadIdx.x & 31;
    for (int64_t base = blockIdx.x; base < units; base += 32 * (int64_t)gridDim.x) {
      const int64_t mine = base + lane * (int64_t)gridDim.x;
      const int m_of = (int)(mine / (per * 2)), part_of = (int)(mine - (int64_t)m_of * (per * 2));
      const int a_of = mine < units ? src[m_of] : -1, b_of = mine < units ? dst[m_of] : -1;
      const bool some = a_of >= 0 && b_of >= 0, bad = some && (a_of >= C.P || b_of >= C.P);
      if (bad) atomicOr(&g_cache_status, kCacheBadPage);
      for (uint32_t left = __ballot_sync(0xffffffffu, some && !bad); left; left &= left - 1) {
        const int who = __ffs(left) - 1;
        const int a = __shfl_sync(0xffffffffu, a_of, who), b = __shfl_sync(0xffffffffu, b_of, who);
        const int part = __shfl_sync(0xffffffffu, part_of, who);
        const Pages &x = part < per ? kp : vp;
        const int first = (part < per ? part : part - per) * kCopyThreads * kCopyInFlight + threadIdx.x;
        uint4 v[kCopyInFlight];
        int64_t at[kCopyInFlight];
#pragma unroll
        for (int i = 0; i < kCopyInFlight; ++i) {
            const int y = first + i * kCopyThreads;
            at[i] = -1;
            if (y < page) {
                if (DENSE) {
                    at[i] = (int64_t)y * 8;
                } else {
                    const int c = y % pieces, h = y / pieces % C.H, t = y / (pieces * C.H);
                    at[i] = t * x.token + h * x.head + c * 8;
                }
                v[i] = *reinterpret_cast<const uint4 *>(x.p + a * x.page + at[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kCopyInFlight; ++i)
            if (at[i] >= 0) *reinterpret_cast<uint4 *>(x.p + b * x.page + at[i]) = v[i];
      }
    }
}

template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), unsigned blocks, int threads, cudaStream_t stream, const Args &...args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t kda_launch_cache_reserve(const Cache &C, const int32_t *new_lens, int32_t *src, int32_t *dst, int32_t *missing,
                                     int32_t *granted, int32_t *list, cudaStream_t stream) {
    kda_cache_reserve_kernel<<<1, kBlock, 0, stream>>>(C, new_lens, src, dst, missing, granted, list);
    return cudaGetLastError();
}

cudaError_t kda_launch_cache_append(const Cache &C, const Heads &k, const Heads &v, const Pages &kp, const Pages &vp,
                                    const int32_t *cu, int64_t T, int64_t seq_len, const int32_t *granted,
                                    cudaStream_t stream) {
    kda_cache_append_kernel<<<(unsigned)((T + kAppendTokens - 1) / kAppendTokens), 256, 0, stream>>>(C, k, v, kp, vp, cu, T,
                                                                                                    seq_len, granted);
    return cudaGetLastError();
}

cudaError_t kda_launch_cache_free(const Cache &C, int M, const int32_t *seqs, const int32_t *keep, cudaStream_t stream) {
    kda_cache_free_kernel<<<(unsigned)M, 256, 0, stream>>>(C, seqs, keep);
    return cudaGetLastError();
}

cudaError_t kda_launch_cache_fork(const Cache &C, int M, const int32_t *parents, const int32_t *children, int32_t *src,
                                  int32_t *dst, int32_t *missing, int32_t *list, cudaStream_t stream) {
    // Few entries: the rows in the same launch.  That saves the host a launch, which is what a call by itself waits for
    // (fork and free of 4 children by 64 entries and of 96 by 70: 19 us a pair against 22).  In a graph the
    // device alone counts, and one block is slower from some 1,500 entries on: 5.9 us a pair against 6.7 for 1 by
    // 64, 7.7 and 8.8 for 16 by 64, 10.3 and 9.5 for 96 by 70, 18.6 and 10.0 for 96 by 512, 16.4 and 9.9 for 512
    // by 16.  The border lies where both lose little.
    const bool rows = (int64_t)M * C.wide <= 8 * kBlock;
    kda_cache_fork_pages_kernel<<<1, kBlock, 0, stream>>>(C, M, parents, children, src, dst, missing, list, rows);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || rows) return e;
    return launch_behind(kda_cache_fork_rows_kernel, (unsigned)M, 256, stream, C, parents, children, (const int32_t *)dst);
}

cudaError_t kda_launch_cache_compact(const Cache &C, int32_t *refs_out, int32_t *table_out, int32_t *src, int32_t *dst,
                                     int32_t *to, cudaStream_t stream) {
    int32_t *counts = to + C.P;
    kda_cache_plan_kernel<<<kCluster, kBlock, 0, stream>>>(C.refs, C.P, src, dst, to, counts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t most = C.P > (int64_t)C.N * C.wide ? C.P : (int64_t)C.N * C.wide;
    const int64_t blocks = (most + 255) / 256;
    return launch_behind(kda_cache_renumber_kernel, (unsigned)(blocks > 1216 ? 1216 : blocks), 256, stream, C,
                         (const int32_t *)src, (const int32_t *)dst, (const int32_t *)to, (const int32_t *)counts, refs_out,
                         table_out);
}

cudaError_t kda_launch_cache_copy(const Cache &C, const Pages &kp, const Pages &vp, int M, const int32_t *src,
                                  const int32_t *dst, cudaStream_t stream) {
    // a page whose elements fill one run of memory is copied as that run
    const auto dense = [&](const Pages &x) {
        const int64_t d = C.d, page = (int64_t)1 << C.shift;
        return (x.head == d || C.H == 1) && (x.token == d * C.H || page == 1)          // tokens, then heads
                   ? true
                   : x.token == d && (x.head == d * page || C.H == 1);                  // heads, then tokens
    };
    const int64_t page = (int64_t)(C.H * (C.d / 8)) << C.shift;
    const int64_t units = (page + kCopyThreads * kCopyInFlight - 1) / (kCopyThreads * kCopyInFlight) * 2 * M;
    const unsigned grid = (unsigned)(units < 152 * 16 ? units : 152 * 16);
    if (dense(kp) && dense(vp))
        kda_cache_copy_kernel<true><<<grid, kCopyThreads, 0, stream>>>(C, kp, vp, M, src, dst);
    else
        kda_cache_copy_kernel<false><<<grid, kCopyThreads, 0, stream>>>(C, kp, vp, M, src, dst);
    return cudaGetLastError();
}

cudaError_t kda_cache_read_status(unsigned *status) {
    unsigned w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&w, g_cache_status, sizeof(w));
    if (e == cudaSuccess && w) {
        *status |= w;
        w = 0;
        e = cudaMemcpyToSymbol(g_cache_status, &w, sizeof(w));
    }
    return e;
}
