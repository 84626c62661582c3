// The accepted path of a drafted tree (contract: focus.h).  A warp a sequence, two nodes
// a lane: a node is accepted when its line lies within the word of the nodes whose token is
// the one that was chosen after their parent.  A launch's latency: 2.6 us for one sequence, 3.6 for 512
// (0.4 MB).
#include "tree.cuh"

namespace focus {
namespace {

constexpr int kWarps = 4;

__global__ void __launch_bounds__(kWarps * 32) tree_accept_kernel(TreeAcceptLaunch L) {
  __shared__ unsigned long long s_line[kWarps][kMaxNodes];
  __shared__ int s_up[kWarps][kMaxNodes];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, b = blockIdx.x * kWarps + warp;
  if (b >= L.B) return;
  int m = L.n;
  if (L.n_new) {
    m = L.n_new[b];
    if (m < 0 || m > L.n) {
      atomicOr(L.err, kErrBadCache);
      m = m < 0 ? 0 : L.n;
    }
  }
  const size_t at = static_cast<size_t>(b) * L.n;
  const int prev = L.prev[b];
  bool right[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    right[i] = false;
    if (t < m) {
      const int p = L.parent[at + t];
      right[i] = L.token[at + t] == (p >= 0 && p < t ? L.target[at + p] : prev);
    }
  }
  unsigned long long* line = s_line[warp];
  tree_lines(L.parent + at, m, line, s_up[warp], L.err);
  const unsigned long long ok = __ballot_sync(~0u, right[0]) | static_cast<unsigned long long>(__ballot_sync(~0u, right[1])) << 32;
  // the deepest accepted node, ties: the lowest index
  int key = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned long long l = line[lane + 32 * i];
    if ((l & ~ok) == 0) key = max(key, __popcll(l) * kMaxNodes + (kMaxNodes - 1 - (lane + 32 * i)));
  }
  key = __reduce_max_sync(~0u, key);
  const int count = key / kMaxNodes, best = kMaxNodes - 1 - key % kMaxNodes;
  const unsigned long long path = count ? line[best] : 0ull;         // its bits rise from the root to the node
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    if (path >> t & 1) L.rows[at + __popcll(path & ((1ull << t) - 1))] = t;
  }
  if (lane == 0) {
    L.count[b] = count;
    L.last[b] = count ? L.target[at + best] : prev;
  }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptLaunch& L, cudaStream_t st) {
  tree_accept_kernel<<<(L.B + kWarps - 1) / kWarps, kWarps * 32, 0, st>>>(L);
  return cudaGetLastError();
}

}  // namespace focus
