// ragged.cuh -- ragged batches: rows row_start[b] .. row_start[b + 1] - 1 belong to request b.
#pragma once

#include "common.cuh"

namespace sd {

// The request that new row t belongs to: the last b with row_start[b] <= t (rs in shared memory).
__device__ __forceinline__ int request_of(const int* rs, int B, int t) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (rs[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// row_start into shared memory, checked: starts at 0 or above, never falls, ends within the batch.
__device__ __forceinline__ bool load_row_start(const int32_t* row_start, int B, int total_rows, int* rs,
                                               int32_t* status) {
    bool bad = false;
    for (int i = threadIdx.x; i <= B; i += blockDim.x) {
        const int v = row_start[i], prev = i > 0 ? row_start[i - 1] : 0;
        bad = bad || v < prev || v > total_rows;
        rs[i] = v;
    }
    if (__syncthreads_or(bad ? 1 : 0)) {
        if (threadIdx.x == 0) report(status, SD_ERR_INVALID_ARG);
        return false;
    }
    return true;
}

}  // namespace sd
