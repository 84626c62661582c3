// Device helpers of the paged 8-bit key/value cache: bounds-checked lookups,
// e4m3 conversions and the page scale rule.
#pragma once

#include <cuda_fp16.h>

#include <atomic>
#include <mutex>

#include "common.cuh"

namespace focus {

// Slots of head h in use, kept inside the table (a bad count raises the flag).
__device__ __forceinline__ int cache_len(const focus_cache_t& c, int H_kv, int b, int h, int* err) {
  const int n = c.len[b * H_kv + h];
  const int cap = c.max_pages * kPage;
  if (n >= 0 && n <= cap) return n;
  atomicOr(err, kErrBadCache);
  return n < 0 ? 0 : cap;
}

// Page j of sequence b, or -1 (and the flag) for an id outside the pool.
__device__ __forceinline__ int cache_page(const focus_cache_t& c, int b, int j, int* err) {
  const int g = c.table[static_cast<size_t>(b) * c.max_pages + j];
  if (g >= 0 && g < c.n_pages) return g;
  atomicOr(err, kErrBadCache);
  return -1;
}

// New tokens of sequence b: n_new[b] inside [0, n] (n without the array).
__device__ __forceinline__ int cache_new(const int32_t* n_new, int n, int b, int* err) {
  if (!n_new) return n;
  const int m = n_new[b];
  if (m >= 0 && m <= n) return m;
  atomicOr(err, kErrBadCache);
  return m < 0 ? 0 : n;
}

// The keep rule: query position i, key position j, window w >= 1.
__device__ __forceinline__ bool cache_keep(int i, int j, int w, bool same_group) {
  return j <= i && (same_group || static_cast<uint32_t>(i) - static_cast<uint32_t>(j) < static_cast<uint32_t>(w));
}

__device__ __forceinline__ float exp2_int(int e) {   // 2^e, -126 <= e <= 127
  return __int_as_float((e + 127) << 23);
}

constexpr int kMaxExp = 120;           // largest exponent that the append writes: fp32 ends below 448 * 2^120

// Exponent of a stored scale, inside the range the append writes.
__device__ __forceinline__ int scale_exp(float s) {
  const int e = static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127;
  return min(max(e, kMinExp), kMaxExp);
}

// Scales of K and V of a page as they are stored, and their exponents in two bytes.
// Kept apart: the bytes are formed when they are needed, not when the loads start.
struct PageScales {
  float k, v;
  __device__ __forceinline__ void load(const focus_cache_t& c, size_t plane) {
    k = c.k_scale[plane];
    v = c.v_scale[plane];
  }
  __device__ __forceinline__ int bytes() const { return (scale_exp(k) & 0xff) | (scale_exp(v) & 0xff) << 8; }
};

// Least e >= least with a <= 448 * 2^e = 1.75 * 2^(e + 8), from the bits of a finite
// a >= 0.  For a page anything below 2^-56 needs no more than kMinExp.
__device__ __forceinline__ int need_exp(uint32_t a, int least = kMinExp) {
  const int x = static_cast<int>(a >> 23) - 127;
  return max(x - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0), least);
}

// Least exponent that a query row is scaled by.  There bf16 numbers, multiples of 2^-133,
// are multiples of 2^-10 and whole in either kernel's parts, fp32 rows of normal numbers
// (2^-3 or more) keep 22 bits in two f16 parts, and the row's factor 2^e * scale * log2(e)
// is still a normal number for the usual scale.
constexpr int kMinQueryExp = -123;

// The attention's running sums.  With t_j = s_j + e_j (log2; e_j the exponent of the
// slot's value page) weights are 2^(t_j - ref) and the sum adds 2^(s_j - ref), which is
// the weight times 2^-e_j: exact, unless the weight itself has fallen below the normals.
// ref lies at most s_max + e_top, so for pages whose exponents are no further than this
// apart that happens only below 2^-34 of the row's largest term.  Where the pages of a
// head that have been scanned differ by more, the sum's terms are exponentials of their
// own (kLift at the kernels keeps them in range for any exponents).
constexpr int kScaleSpan = 96;
constexpr float kNoRef = -1e30f;       // reference of a row without kept slots

__device__ __forceinline__ float exp2_fast(float x) {   // 2^x, results below the normals are 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two e4m3 codes (low byte first) <-> floats.  e4m3 fits f16 exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
  const uint32_t r = e4m3x2_to_f16x2(c);
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}
// Round to nearest even, values past 448 to +-448, NaN to NaN.
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sixteen codes times 2^d, rounded to e4m3 again.  For |d| <= 14 the product is
// exact in f16 (codes are multiples of 2^-9, f16's least is 2^-24; results that
// overflow saturate either way), so only the rounding to e4m3 rounds.
__device__ __forceinline__ uint4 rescale16(uint4 c, int d) {
  uint32_t w[4] = {c.x, c.y, c.z, c.w};
  if (d >= -14 && d <= 14) {
    const __half2 f = __half2half2(__ushort_as_half(static_cast<uint16_t>((d + 15) << 10)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t r[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t x = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> (16 * e)));
        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x), f);
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r[e]) : "r"(*reinterpret_cast<const uint32_t*>(&y)));
      }
      w[i] = r[0] | static_cast<uint32_t>(r[1]) << 16;
    }
  } else {
    const float f = exp2_int(min(max(d, -126), 127));        // codes times 2^-126 are 0 like any smaller factor
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(w[i]));
      const float2 b = e4m3x2_to_float2(static_cast<uint16_t>(w[i] >> 16));
      w[i] = float2_to_e4m3x2(a.x * f, a.y * f) | static_cast<uint32_t>(float2_to_e4m3x2(b.x * f, b.y * f)) << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude code of sixteen, NaN left out.
__device__ __forceinline__ uint32_t top_code(uint4 c) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t lo = 0, hi = 0;                                   // bytes 0 and 2, 1 and 3, a pair of maxima each
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo = __vmaxu2(lo, w[i] & 0x007f007fu);
    hi = __vmaxu2(hi, w[i] & 0x7f007f00u);
  }
  uint32_t top = max(max(lo & 0xffffu, lo >> 16), max(hi & 0xffffu, hi >> 16) >> 8);
  if (top == 127) {
    top = 0;
    for (int i = 0; i < 16; ++i) {
      const uint32_t x = w[i / 4] >> (i % 4 * 8) & 127u;
      if (x < 127) top = max(top, x);
    }
  }
  return top;
}

// Clusters of 1, 2, 4, 8 and 16 blocks of a kernel that a device runs at once.  A
// cluster lies within one part of the GPU and the parts differ in SMs, so these are
// fewer than the SMs hold blocks: with one block an SM, 16 blocks a cluster leave so
// many SMs over that eight clusters take two waves.
struct ClusterFit {
  int n[5];
};
constexpr int kMaxClusterBlocks = 16;

inline cudaError_t cluster_fit(const void* kernel, int threads, size_t smem, ClusterFit* fit) {
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem))) return e;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) return e;
  for (int i = 0; i < 5; ++i) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1 << i);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1 << i;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaError_t e = cudaOccupancyMaxActiveClusters(&fit->n[i], kernel, &cfg)) return e;
  }
  return cudaSuccess;
}

// A kernel's attributes and cluster figures per device, asked for at its first launch
// there: a program that makes no such call loads no such kernel.
class ClusterFits {
 public:
  cudaError_t get(int device, const void* kernel, int threads, size_t smem, const ClusterFit** fit) {
    if (!ready_[device].load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mu_);
      if (!ready_[device].load(std::memory_order_relaxed)) {
        if (cudaError_t e = cluster_fit(kernel, threads, smem, &fit_[device])) return e;
        ready_[device].store(true, std::memory_order_release);
      }
    }
    *fit = &fit_[device];
    return cudaSuccess;
  }

 private:
  std::mutex mu_;
  std::atomic<bool> ready_[kMaxDevices] = {};
  ClusterFit fit_[kMaxDevices];
};

}  // namespace focus
