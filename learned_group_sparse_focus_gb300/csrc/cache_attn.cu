// Focus attention of new tokens over the paged 8-bit cache (contract: focus.h).
//
// One block per (sequence, key/value head): its eight warps share the pages,
// each warp runs an online softmax over its kept slots, and the block joins the
// eight partial results.
#include "cache.cuh"

namespace focus {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) cache_attn_kernel(CacheAttnLaunch L) {
  constexpr int kDims = D / 32;               // dims a lane holds
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int h = blockIdx.x, b = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = L.H / (L.H_kv);
  const int n = cache_len(L.c, L.H_kv, b, h, L.err);
  const int fresh = cache_new(L.n_new, L.n, b, L.err);
  const int pages = (n + kPage - 1) / kPage;
  for (int t = 0; t < fresh; ++t) {
    const int pos = L.c.next[b] - fresh + t;
    const int gid = L.gid[(static_cast<size_t>(b) * L.A + (L.A == 1 ? 0 : h)) * L.n + t];
    for (int g = 0; g < G; ++g) {
      const size_t row = (static_cast<size_t>(b) * L.H + h * G + g) * L.n + t;
      float q[kDims], o[kDims] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
      for (int e = 0; e < kDims; ++e)
        q[e] = to_float(static_cast<const T*>(L.Q)[row * D + lane * kDims + e]) * L.scale_log2;
      float lse2 = 0.f;
      for (int pass = 0; pass < (L.logits ? 2 : 1); ++pass) {
        for (int j = warp; j < pages; j += kWarps) {
          const int page = cache_page(L.c, b, j, L.err);
          if (page < 0) continue;
          const size_t plane = static_cast<size_t>(page) * L.H_kv + h;
          const float ks = L.c.k_scale[plane], vs = L.c.v_scale[plane];
          for (int r = 0; r < min(kPage, n - j * kPage); ++r) {
            if (!cache_keep(pos, L.c.pos[plane * kPage + r], L.w, L.c.gid[plane * kPage + r] == gid)) continue;
            const size_t at = (plane * kPage + r) * D + lane * kDims;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < kDims; ++e) s += q[e] * e4m3x2_to_float2(L.c.k[at + e]).x;
#pragma unroll
            for (int x = 16; x > 0; x /= 2) s += __shfl_xor_sync(~0u, s, x);
            s *= ks;
            if (pass == 1) {
              if (lane == 0) L.c.mass[plane * kPage + r] += exp2f(s - lse2);
              continue;
            }
            const float top = fmaxf(m, s), c = exp2f(m - top), p = exp2f(s - top);
            m = top;
            l = l * c + p;
#pragma unroll
            for (int e = 0; e < kDims; ++e) o[e] = o[e] * c + p * vs * e4m3x2_to_float2(L.c.v[at + e]).x;
          }
        }
        if (pass == 1) break;
        if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
        for (int e = 0; e < kDims; ++e) s_o[warp][lane * kDims + e] = o[e];
        __syncthreads();
        float top = -INFINITY, total = 0.f;
        for (int i = 0; i < kWarps; ++i) top = fmaxf(top, s_m[i]);
        for (int i = 0; i < kWarps; ++i) total += s_l[i] != 0.f ? s_l[i] * exp2f(s_m[i] - top) : 0.f;
        if (threadIdx.x < D) {
          float x = 0.f;
          for (int i = 0; i < kWarps; ++i)
            x += s_l[i] != 0.f ? s_o[i][threadIdx.x] * exp2f(s_m[i] - top) : 0.f;
          store(static_cast<T*>(L.O) + row * D + threadIdx.x, total != 0.f ? x / total : 0.f);
        }
        lse2 = top + log2f(total);
        if (threadIdx.x == 0 && L.lse)
          L.lse[row] = total != 0.f ? lse2 * 0.6931471805599453f : -INFINITY;
        __syncthreads();
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnLaunch& L, int dtype, cudaStream_t st) {
  const dim3 grid(L.H_kv, L.B);
  if (dtype == FOCUS_BF16) {
    if (L.d == 128) cache_attn_kernel<__nv_bfloat16, 128><<<grid, kWarps * 32, 0, st>>>(L);
    else cache_attn_kernel<__nv_bfloat16, 64><<<grid, kWarps * 32, 0, st>>>(L);
  } else {
    if (L.d == 128) cache_attn_kernel<float, 128><<<grid, kWarps * 32, 0, st>>>(L);
    else cache_attn_kernel<float, 64><<<grid, kWarps * 32, 0, st>>>(L);
  }
  return cudaGetLastError();
}

}  // namespace focus
