// kda_api_util.cuh -- argument checks shared by the C entry points.
#pragma once

#include <initializer_list>

#include "kda_common.cuh"

// Records the error's text for kda_last_cuda_error and returns KDA_ERR_CUDA.
kda_status kda_cuda_fail(cudaError_t e, const char *where);

namespace kda {

// Do the byte ranges [a, a + na) and [b, b + nb) share a byte?
inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const char *x = (const char *)a, *y = (const char *)b;
    return x < y + nb && y < x + na;
}

// A buffer a call touches: its address and size in bytes (a NULL buffer is empty).
struct Span {
    const void *p;
    size_t n;
};

// Does a written buffer share a byte with a read buffer or with another
// written buffer?  The kernels read inputs (some by TMA, chunks ahead) while
// they write outputs, so any such overlap would be a race.
inline bool conflict(std::initializer_list<Span> writes, std::initializer_list<Span> reads) {
    for (const Span *w = writes.begin(); w != writes.end(); ++w) {
        for (const Span &r : reads)
            if (overlaps(w->p, w->n, r.p, r.n)) return true;
        for (const Span *w2 = w + 1; w2 != writes.end(); ++w2)
            if (overlaps(w->p, w->n, w2->p, w2->n)) return true;
    }
    return false;
}

inline size_t esize(int32_t dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

inline bool valid_dtype(int32_t d) { return d == KDA_DTYPE_F32 || d == KDA_DTYPE_BF16; }

}  // namespace kda
