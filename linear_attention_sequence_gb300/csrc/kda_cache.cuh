// kda_cache.cuh -- the cache as the page kernels see it, and their launchers.
#pragma once

#include "kda_common.cuh"

namespace kda {

// The bookkeeping of a cache; pages hold 2^shift tokens of H heads by d channels (16-bit).
struct Cache {
    int32_t N, P, wide, shift, H, d;
    int32_t *refs;    // [P]
    int32_t *table;   // [N, wide]
    int32_t *lens;    // [N]
};
// 16-bit elements with strides.
struct Heads {
    const uint16_t *p;
    int64_t token, head;
};
struct Pages {
    uint16_t *p;
    int64_t page, token, head;
};

}  // namespace kda

cudaError_t kda_launch_cache_reserve(const kda::Cache &C, const int32_t *new_lens, int32_t *src, int32_t *dst, int32_t *missing,
                                     int32_t *granted, int32_t *list, cudaStream_t stream);
cudaError_t kda_launch_cache_append(const kda::Cache &C, const kda::Heads &k, const kda::Heads &v, const kda::Pages &kp,
                                    const kda::Pages &vp, const int32_t *cu, int64_t T, int64_t seq_len, const int32_t *granted,
                                    cudaStream_t stream);
cudaError_t kda_launch_cache_free(const kda::Cache &C, int M, const int32_t *seqs, const int32_t *keep, cudaStream_t stream);
cudaError_t kda_launch_cache_fork(const kda::Cache &C, int M, const int32_t *parents, const int32_t *children, int32_t *src,
                                  int32_t *dst, int32_t *missing, int32_t *list, cudaStream_t stream);
cudaError_t kda_launch_cache_compact(const kda::Cache &C, int32_t *refs_out, int32_t *table_out, int32_t *src, int32_t *dst,
                                     int32_t *to, cudaStream_t stream);
cudaError_t kda_launch_cache_copy(const kda::Cache &C, const kda::Pages &kp, const kda::Pages &vp, int M, const int32_t *src,
                                  const int32_t *dst, cudaStream_t stream);
