// topk.cuh -- the top-k step shared by the routing kernels.
#pragma once

#include "plan.h"

namespace moe {

__device__ __forceinline__ float finite_or_minus_inf(float v) { return v != v ? -INFINITY : v; }

// Inserts (v, e) into a descending list of at most k entries held in
// registers; a larger value goes first, an equal one after the entries
// already there (experts arrive in increasing index, so the lower index keeps
// a tie).  From the insertion point on every entry shifts down one place and
// the old k-th falls off.
__device__ __forceinline__ void topk_insert(float* val, int* id, int k, float v, int e) {
    if (!(id[k - 1] < 0 || v > val[k - 1])) return;
    float cv = v;
    int ci = e;
    bool ins = false;
#pragma unroll
    for (int q = 0; q < MAX_K; ++q) {
        if (q < k && (ins || id[q] < 0 || cv > val[q])) {
            const float tv = val[q];
            const int ti = id[q];
            val[q] = cv;
            id[q] = ci;
            cv = tv;
            ci = ti;
            ins = true;
        }
    }
}

}  // namespace moe
