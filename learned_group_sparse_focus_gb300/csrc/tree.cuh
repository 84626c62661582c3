// Trees of drafted tokens (contract: focus.h): up to 64 nodes a sequence, so a node's
// line, itself and its ancestors, is a 64-bit word.
#pragma once

#include "common.cuh"

namespace focus {

constexpr int kMaxNodes = FOCUS_CACHE_MAX_QUERY;
static_assert(kMaxNodes == 64, "lines are 64-bit words");

// Lines of the first m nodes of a tree, by one whole warp, into shared memory: each round
// doubles the steps towards the root that a line holds.  A parent that is not -1 or an earlier
// node raises the flag and counts as -1.
__device__ __forceinline__ void tree_lines(const int32_t* parent, int m, unsigned long long* line, int* up, int* err) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    int p = -1;
    if (t < m) {
      p = parent[t];
      if (p < -1 || p >= t) {
        atomicOr(err, kErrBadTree);
        p = -1;
      }
    }
    line[t] = 1ull << t;
    up[t] = p;
  }
  __syncwarp();
#pragma unroll
  for (int step = 1; step < kMaxNodes; step *= 2) {
    unsigned long long l[2];
    int p[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = lane + 32 * i;
      l[i] = line[t];
      p[i] = up[t];
      if (p[i] >= 0) {
        l[i] |= line[p[i]];
        p[i] = up[p[i]];
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      line[lane + 32 * i] = l[i];
      up[lane + 32 * i] = p[i];
    }
    __syncwarp();
  }
}

}  // namespace focus
