// Shared by the kernels of the paged cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace lin {

// The sequence that row n belongs to: the last b with q_start[b] <= n, or -1. By one
// warp, 32 entries a step. q_start[0 .. B) is read and nothing else, whatever it holds.
__device__ __forceinline__ int find_sequence(const int* q_start, int B, int n) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = B;
    while (hi - lo > 32) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const int c = __popc(__ballot_sync(0xffffffffu, i < hi && q_start[i] <= n));
        if (c == 0) return -1;
        lo += (c - 1) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    const int c = __popc(__ballot_sync(0xffffffffu, lo + lane < hi && q_start[lo + lane] <= n));
    return c == 0 ? -1 : lo + c - 1;
}

}  // namespace lin
