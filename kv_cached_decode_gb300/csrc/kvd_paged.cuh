// kvd_paged.cuh -- the packed ragged batch and the page table, for the kernels over a paged cache.
#pragma once

#include "kvd_common.cuh"
#include "kvd_internal.h"

namespace kvd {

// Positions a row of the table can hold; sums of positions stay in 32 bits.
constexpr int64_t kPagedMaxLen = INT64_C(1) << 30;

// Row b's new tokens are starts[b] .. starts[b+1]-1 of n_tokens packed ones. Whether that is a
// stretch of the packed tokens; n receives its length.
__device__ __forceinline__ bool row_tokens(const int32_t* starts, int b, int n_tokens, int& s,
                                           int& n) {
    s = starts[b];
    const int e = starts[b + 1];
    const bool ok = s >= 0 && e >= s && e <= n_tokens;
    n = ok ? e - s : 0;
    return ok;
}

// The row that holds packed token t: the last one that starts at or before it. All lanes of a
// warp together, 32 rows a step; some row in [0, batch) whatever `starts` holds.
__device__ __forceinline__ int find_token_row(const int32_t* starts, int batch, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const unsigned before = __ballot_sync(0xffffffffu, at < hi && starts[at] <= t);
        // (a lane past a gap counts only in a `starts` that is not ascending)
        const int k = __ffs(~before) - 1;
        lo += (k < 0 ? 32 : k) * step;
        hi = min(lo + step, hi);
    }
    return lo;
}

}  // namespace kvd
