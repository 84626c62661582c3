// Paged 8-bit key/value cache: append and eviction (contract: focus.h).
//
// Both move rows once and are bound by HBM: the append reads 2 d elements of
// the model's type a token and head and writes 2 d codes, the eviction reads
// and writes 2 d codes a kept slot, after a selection that reads 4 bytes of
// mass a slot.
//
// The page scale is a power of two.  e4m3 keeps a relative step of 2^-3 over
// its whole normal range, so a finer scale gains no accuracy there, and with a
// power of two every scaling is exact: x * 2^-e is rounded once, to e4m3.
#include "cache.cuh"

namespace focus {
namespace {

constexpr int kThreads = 256;
constexpr int kHalf = kThreads / 2;    // the first half moves K, the second V

// ----------------------------------------------------------------- append ---

// Eight consecutive elements of a row as floats.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Whether m more tokens fit every head of sequence b (same answer in all
// threads of the block; contains a block barrier).
__device__ __forceinline__ bool sequence_fits(const CacheAppendLaunch& L, int b, int m) {
  const int cap = L.c.max_pages * kPage;
  bool ok = L.c.next[b] >= 0 && L.c.next[b] <= 0x7fffffff - m;
  for (int h = threadIdx.x; h < L.H_kv; h += kThreads) {
    const int n = L.c.len[b * L.H_kv + h];
    ok = ok && n >= 0 && n <= cap - m;
  }
  return __syncthreads_and(ok);
}

// One block per touched page and head: the new rows of the page stay in
// registers between the search for the largest magnitude and the rounding, so
// they are read once.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(CacheAppendLaunch L) {
  constexpr int kPerRow = D / 8;                       // 8-element pieces of a row
  constexpr int kPieces = kPage * kPerRow / kHalf;     // pieces a thread holds
  __shared__ uint32_t s_max[kThreads / 32];
  __shared__ int s_last;
  const int b = blockIdx.z, h = blockIdx.y;
  const int half = threadIdx.x / kHalf, ht = threadIdx.x % kHalf;
  const int m = cache_new(L.n_new, L.n, b, L.err);
  const bool fits = sequence_fits(L, b, m);
  const int n0 = L.c.len[b * L.H_kv + h];
  if (!fits && threadIdx.x == 0) atomicOr(L.err, kErrBadCache);
  const int j = n0 / kPage + blockIdx.x;
  const int lo = max(n0, j * kPage), hi = min(n0 + m, (j + 1) * kPage);
  const int page = fits && lo < hi ? cache_page(L.c, b, j, L.err) : -1;
  if (page >= 0) {
    const int r0 = lo - j * kPage, rows = hi - lo, t0 = lo - n0;
    const size_t plane = static_cast<size_t>(page) * L.H_kv + h;
    const T* src = static_cast<const T*>(half ? L.V : L.K) +
                   ((static_cast<size_t>(b) * L.H_kv + h) * L.n + t0) * D;
    uint8_t* dst = (half ? L.c.v : L.c.k) + plane * kPage * D;
    float* scale = (half ? L.c.v_scale : L.c.k_scale) + plane;
    float x[kPieces][8];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = ht + i * kHalf;
      if (at >= rows * kPerRow) continue;
      load8(src + static_cast<size_t>(at) * 8, x[i]);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (ht + i * kHalf >= rows * kPerRow) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = __float_as_uint(x[i][e]) & 0x7fffffffu;
        if (u < 0x7f800000u) a = max(a, u);
      }
    }
    const int e_old = r0 > 0 ? scale_exp(*scale) : kMinExp;
    a = __reduce_max_sync(~0u, a);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHalf / 32; ++i) a = max(a, s_max[half * (kHalf / 32) + i]);
    const int e = max(need_exp(a), e_old);
    if (ht == 0) *scale = exp2_int(e);
    if (e > e_old) {                                   // the page's older rows, at the new scale
      const float f = exp2_int(max(e_old - e, -126));  // codes times 2^-126 are 0 like any smaller factor
      uint4* old = reinterpret_cast<uint4*>(dst);
      for (int at = ht; at < r0 * D / 16; at += kHalf) old[at] = rescale16(old[at], f);
    }
    const float f = exp2_int(-e);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = ht + i * kHalf;
      if (at >= rows * kPerRow) continue;
      uint32_t w[2];
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        const float* y = x[i] + 4 * e2;
        w[e2] = static_cast<uint32_t>(float2_to_e4m3x2(y[0] * f, y[1] * f)) |
                (static_cast<uint32_t>(float2_to_e4m3x2(y[2] * f, y[3] * f)) << 16);
      }
      *reinterpret_cast<uint2*>(dst + static_cast<size_t>(r0) * D + static_cast<size_t>(at) * 8) =
          make_uint2(w[0], w[1]);
    }
    if (ht < rows) {
      const size_t at = plane * kPage + r0 + ht;
      if (half == 0) {
        int g = L.gid[(static_cast<size_t>(b) * L.A + (L.A == 1 ? 0 : h)) * L.n + t0 + ht];
        if (g < 0 || g >= L.K_groups) {
          atomicOr(L.err, kErrBadGroup);
          g = g < 0 ? 0 : L.K_groups - 1;
        }
        L.c.pos[at] = L.c.next[b] + t0 + ht;
        L.c.gid[at] = static_cast<int16_t>(g);
      } else if (L.c.mass) {
        L.c.mass[at] = 0.f;
      }
    }
  }
  // The last block to finish writes the new counts: by then every block has
  // read the old ones, so they may be updated in place.
  __syncthreads();
  if (threadIdx.x == 0) {
    const int total = gridDim.x * gridDim.y * gridDim.z;
    __threadfence();
    s_last = atomicAdd(L.ticket, 1) == total - 1;
  }
  __syncthreads();
  if (!s_last) return;
  const int cap = L.c.max_pages * kPage;
  for (int s = threadIdx.x / 32; s < L.B; s += kThreads / 32) {   // a warp a sequence
    const int lane = threadIdx.x % 32;
    const int more = cache_new(L.n_new, L.n, s, L.err), next = L.c.next[s];
    bool ok = next >= 0 && next <= 0x7fffffff - more;
    for (int i = lane; i < L.H_kv; i += 32) {
      const int n = L.c.len[s * L.H_kv + i];
      ok = ok && n >= 0 && n <= cap - more;
    }
    const int add = __all_sync(~0u, ok) ? more : 0;
    for (int i = lane; i < L.H_kv; i += 32) L.len_out[s * L.H_kv + i] = L.c.len[s * L.H_kv + i] + add;
    if (lane == 0) L.next_out[s] = next + add;
  }
  if (threadIdx.x == 0) *L.ticket = 0;
}

// --------------------------------------------------------------- eviction ---

// Order of the slots an eviction may drop: larger keys stay.  Mass ascending
// (-0 as 0), NaN above every number, protected slots above all.
__device__ __forceinline__ uint32_t keep_key(float mass, bool late) {
  if (late) return 0xffffffffu;
  const uint32_t u = __float_as_uint(mass);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xfffffffeu;
  if (u == 0x80000000u) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;

__device__ __forceinline__ uint32_t slot_key(const CacheEvictLaunch& L, int b, int h, int s, int first_late) {
  const int page = cache_page(L.src, b, s / kPage, L.err);
  if (page < 0) return 0;
  const size_t at = (static_cast<size_t>(page) * L.H_kv + h) * kPage + s % kPage;
  return keep_key(L.src.mass[at], L.src.pos[at] >= first_late);
}

// One block per (sequence, head): the budget-th largest key by four passes of
// 8-bit counting, then the kept slots in order (ties: the lowest slots).
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(CacheEvictLaunch L) {
  __shared__ int hist[256];
  __shared__ int s_warp[2][kSelThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int n = cache_len(L.src, L.H_kv, b, h, L.err);
  const int next = L.src.next[b];
  int32_t* keep = L.keep + (static_cast<size_t>(b) * L.H_kv + h) * (static_cast<size_t>(L.src.max_pages) * kPage + 1);
  const int kept = min(n, L.budget);
  const int first_late = next - L.recent;
  uint32_t thr = 0;
  int ties = 0;                       // slots equal to the threshold that stay
  if (n > L.budget) {
    if (tid == 0) { s_prefix = 0; s_left = L.budget; }
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      for (int s = tid; s < n; s += kSelThreads) {
        const uint32_t k = slot_key(L, b, h, s, first_late);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = s_left, d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        s_left = left;
        s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
      }
      __syncthreads();
    }
    thr = s_prefix;
    ties = s_left;
  }
  int base = 0, seen = 0;             // kept and tied slots before this round
  for (int s0 = 0; s0 < n; s0 += kSelThreads) {
    const int s = s0 + tid;
    const uint32_t k = s < n ? (n > L.budget ? slot_key(L, b, h, s, first_late) : 1u) : 0u;
    const bool tie = s < n && n > L.budget && k == thr;
    const uint32_t lanes_before = (1u << (tid & 31)) - 1;
    const uint32_t tb = __ballot_sync(~0u, tie);
    if ((tid & 31) == 0) s_warp[0][tid / 32] = __popc(tb);
    __syncthreads();
    int tie_rank = seen + __popc(tb & lanes_before), tie_sum = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < tid / 32) tie_rank += s_warp[0][w];
      tie_sum += s_warp[0][w];
    }
    const bool stay = s < n && (k > thr || (tie && tie_rank < ties));
    const uint32_t kb = __ballot_sync(~0u, stay);
    if ((tid & 31) == 0) s_warp[1][tid / 32] = __popc(kb);
    __syncthreads();
    int rank = base + __popc(kb & lanes_before), sum = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < tid / 32) rank += s_warp[1][w];
      sum += s_warp[1][w];
    }
    if (stay && rank < kept) keep[1 + rank] = s;
    base += sum;
    seen += tie_sum;
    __syncthreads();
  }
  if (tid == 0) {
    keep[0] = kept;
    L.dst.len[b * L.H_kv + h] = kept;
    if (h == 0) L.dst.next[b] = next;
  }
}

// One block per destination page and head.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_copy_kernel(CacheEvictLaunch L) {
  constexpr int kPerRow = D / 16;
  constexpr int kPieces = kPage * kPerRow / kHalf;
  __shared__ int s_max[kThreads / 32];
  const int j = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int half = threadIdx.x / kHalf, ht = threadIdx.x % kHalf;
  const int32_t* keep = L.keep + (static_cast<size_t>(b) * L.H_kv + h) * (static_cast<size_t>(L.src.max_pages) * kPage + 1);
  const int rows = min(keep[0] - j * kPage, kPage);
  if (rows <= 0) return;
  const int to = cache_page(L.dst, b, j, L.err);
  if (to < 0) return;
  const size_t to_plane = static_cast<size_t>(to) * L.H_kv + h;
  uint4 c[kPieces];
  int es[kPieces];
  int e = kMinExp;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = ht + i * kHalf;
    c[i] = make_uint4(0, 0, 0, 0);
    es[i] = kMinExp;
    if (at >= rows * kPerRow) continue;
    const int s = keep[1 + j * kPage + at / kPerRow];
    const int page = cache_page(L.src, b, s / kPage, L.err);
    if (page < 0) continue;
    const size_t plane = static_cast<size_t>(page) * L.H_kv + h;
    c[i] = *reinterpret_cast<const uint4*>((half ? L.src.v : L.src.k) + (plane * kPage + s % kPage) * D +
                                           (at % kPerRow) * 16);
    es[i] = scale_exp((half ? L.src.v_scale : L.src.k_scale)[plane]);
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    uint32_t top = 0;                       // largest magnitude code of each byte lane, NaN left out
    const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t a = w[x] & 0x7f7f7f7fu;
      top = __vmaxu4(top, a & ~__vcmpeq4(a, 0x7f7f7f7fu));
    }
    top = max(max(top & 255u, (top >> 8) & 255u), max((top >> 16) & 255u, top >> 24));
    const float v = e4m3x2_to_float2(static_cast<uint16_t>(top)).x * exp2_int(es[i]);
    e = max(e, need_exp(__float_as_uint(v)));
  }
  e = __reduce_max_sync(~0u, e);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = e;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHalf / 32; ++i) e = max(e, s_max[half * (kHalf / 32) + i]);
  uint8_t* dst = (half ? L.dst.v : L.dst.k) + to_plane * kPage * D;
  if (ht == 0) (half ? L.dst.v_scale : L.dst.k_scale)[to_plane] = exp2_int(e);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = ht + i * kHalf;
    if (at >= rows * kPerRow) continue;
    if (es[i] != e) c[i] = rescale16(c[i], exp2_int(min(max(es[i] - e, -126), 127)));
    *reinterpret_cast<uint4*>(dst + static_cast<size_t>(at) * 16) = c[i];
  }
  if (ht < rows) {
    const int s = keep[1 + j * kPage + ht];
    const int page = cache_page(L.src, b, s / kPage, L.err);
    const size_t from = (static_cast<size_t>(max(page, 0)) * L.H_kv + h) * kPage + s % kPage;
    const size_t at = to_plane * kPage + ht;
    if (page >= 0 && half == 0) {
      L.dst.pos[at] = L.src.pos[from];
      L.dst.gid[at] = L.src.gid[from];
    } else if (page >= 0) {
      L.dst.mass[at] = L.src.mass[from];
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendLaunch& L, int dtype, cudaStream_t st) {
  // n new slots from anywhere in a page touch at most this many pages
  const dim3 grid((L.n + kPage - 2) / kPage + 1, L.H_kv, L.B);
  if (dtype == FOCUS_BF16) {
    if (L.d == 128) cache_append_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, st>>>(L);
    else cache_append_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, st>>>(L);
  } else {
    if (L.d == 128) cache_append_kernel<float, 128><<<grid, kThreads, 0, st>>>(L);
    else cache_append_kernel<float, 64><<<grid, kThreads, 0, st>>>(L);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const CacheEvictLaunch& L, cudaStream_t st) {
  cache_select_kernel<<<dim3(L.H_kv, L.B), kSelThreads, 0, st>>>(L);
  if (cudaError_t e = cudaGetLastError()) return e;
  const int cap = min(L.budget, L.src.max_pages * kPage);
  const dim3 grid((cap + kPage - 1) / kPage, L.H_kv, L.B);
  if (L.d == 128) cache_copy_kernel<128><<<grid, kThreads, 0, st>>>(L);
  else cache_copy_kernel<64><<<grid, kThreads, 0, st>>>(L);
  return cudaGetLastError();
}

}  // namespace focus
