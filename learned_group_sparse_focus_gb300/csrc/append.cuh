// What the two appends to the paged cache share (cache.cu: rows as they come;
// rotary.cu: keys turned to their positions on the way).
#pragma once

#include "cache.cuh"

namespace focus {

constexpr int kAppendThreads = 256;

// Eight consecutive elements of a row as they are stored, and what the append
// asks of them.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ float at(int e) const {
    const uint32_t w = (&u.x)[e / 2];
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
  }
  // Largest magnitude, as the bits of a float; infinities and NaN included.
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t a = __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
    return max(a & 0xffff0000u, a << 16);
  }
};
template <>
struct Piece<float> {
  uint4 u[2];
  __device__ __forceinline__ void load(const float* p) {
    u[0] = reinterpret_cast<const uint4*>(p)[0];
    u[1] = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = u[0];
    reinterpret_cast<uint4*>(p)[1] = u[1];
  }
  __device__ __forceinline__ float at(int e) const { return __uint_as_float((&u[e / 4].x)[e % 4]); }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t a = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = max(a, (&u[e / 4].x)[e % 4] & 0x7fffffffu);
    return a;
  }
};

// Whether m more tokens fit every head of sequence b (same answer in all lanes
// of a warp).
__device__ __forceinline__ bool sequence_fits(const CacheAppendLaunch& L, int b, int m) {
  const int cap = L.c.max_pages * kPage, next = L.c.next[b];
  bool ok = next >= 0 && next <= 0x7fffffff - m;
  for (int h = threadIdx.x % 32; h < L.H_kv; h += 32) {
    const int n = L.c.len[b * L.H_kv + h];
    ok = ok && n >= 0 && n <= cap - m;
  }
  return __all_sync(~0u, ok);
}

// The counts behind an append; every thread of every block calls it last.  add: tokens
// that (b, h) gained, first: this block writes for (b, h).  Counts that go to other
// arrays are written at once.  Counts updated in place are written by the last block
// to finish: every block has used the old ones by then (a value that has come back
// cannot change, so the ticket needs no fence).
__device__ __forceinline__ void append_counts(const CacheAppendLaunch& L, int b, int h, int n0, int add, bool first,
                                              uint32_t blocks) {
  __shared__ int s_last;
  if (L.len_out != L.c.len && L.next_out != L.c.next) {
    if (first && threadIdx.x == 0) {
      L.len_out[b * L.H_kv + h] = n0 + add;
      if (h == 0) L.next_out[b] = L.c.next[b] + add;
    }
    return;
  }
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(L.ticket, 1) == static_cast<int>(blocks) - 1;
  __syncthreads();
  if (!s_last) return;
  for (int s = threadIdx.x / 32; s < L.B; s += kAppendThreads / 32) {   // a warp a sequence
    const int lane = threadIdx.x % 32;
    const int more = cache_new(L.n_new, L.n, s, L.err);
    const int grown = sequence_fits(L, s, more) ? more : 0;
    for (int i = lane; i < L.H_kv; i += 32) L.len_out[s * L.H_kv + i] = L.c.len[s * L.H_kv + i] + grown;
    if (lane == 0) L.next_out[s] = L.c.next[s] + grown;
  }
  if (threadIdx.x == 0) *L.ticket = 0;
}

}  // namespace focus
