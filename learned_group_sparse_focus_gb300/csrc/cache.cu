// Paged 8-bit key/value cache: append and eviction (contract: focus.h).
//
// Both move rows once and are bound by HBM: the append reads 2 d elements of
// the model's type a token and head and writes 2 d codes, the eviction reads
// and writes 2 d codes a kept slot, after a selection that reads 4 bytes of
// mass a slot.  Measured: 32K tokens of 8 heads, d = 128, bf16 (205 MB) 34 us, 6.0
// TB/s of the 6.8 that a copy reaches; one token for 8 sequences 3.5 us, a launch.
// Eviction of 16 sequences of 8,704 slots, 8 heads, to 8,192 (562 MB) 119 us, 20 of
// them the selection and 99 the copy (5.6 TB/s); 32K slots of one sequence to 4,096,
// 21 us: 16 of the selection's chain of four counting passes over a cluster, 5 of
// the copy.
//
// The page scale is a power of two.  e4m3 keeps a relative step of 2^-3 over
// its whole normal range, so a finer scale gains no accuracy there, and with a
// power of two every scaling is exact: x * 2^-e is rounded once, to e4m3.
#include <cooperative_groups.h>

#include "cache.cuh"

namespace cg = cooperative_groups;

namespace focus {
namespace {

constexpr int kThreads = 256;
constexpr int kHalf = kThreads / 2;    // the first half moves K, the second V

// ----------------------------------------------------------------- append ---

// Eight consecutive elements of a row as they are stored, and what the append
// asks of them.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
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

// One block per touched page and head: the new rows of the page stay in
// registers between the search for the largest magnitude and the rounding, so
// they are read once.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(CacheAppendLaunch L) {
  constexpr int kPerRow = D / 8;                       // pieces of a row
  constexpr int kPieces = kPage * kPerRow / kHalf;     // pieces a thread holds
  __shared__ uint32_t s_max[kThreads / 32];
  __shared__ int s_last;
  const int b = blockIdx.z, h = blockIdx.y;
  const int half = threadIdx.x / kHalf, ht = threadIdx.x % kHalf;
  const int n0 = L.c.len[b * L.H_kv + h];
  const int m = cache_new(L.n_new, L.n, b, L.err);
  const bool fits = sequence_fits(L, b, m);
  if (!fits && threadIdx.x == 0) atomicOr(L.err, kErrBadCache);
  const int j = n0 / kPage + blockIdx.x;
  const int lo = max(n0, j * kPage), hi = min(n0 + m, (j + 1) * kPage);
  if (fits && lo < hi) {
    const int r0 = lo - j * kPage, rows = hi - lo, t0 = lo - n0;
    const T* src = static_cast<const T*>(half ? L.V : L.K) +
                   ((static_cast<size_t>(b) * L.H_kv + h) * L.n + t0) * D;
    Piece<T> x[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (ht + i * kHalf < rows * kPerRow) x[i].load(src + static_cast<size_t>(ht + i * kHalf) * 8);
    const int page = cache_page(L.c, b, j, L.err);
    const size_t plane = static_cast<size_t>(max(page, 0)) * L.H_kv + h;
    float* scale = (half ? L.c.v_scale : L.c.k_scale) + plane;
    const int e_old = r0 > 0 && page >= 0 ? scale_exp(*scale) : kMinExp;
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (ht + i * kHalf < rows * kPerRow) {
        uint32_t top = x[i].top();
        if (top >= 0x7f800000u) {                      // infinities and NaN do not count
          top = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t u = __float_as_uint(x[i].at(e)) & 0x7fffffffu;
            if (u < 0x7f800000u) top = max(top, u);
          }
        }
        a = max(a, top);
      }
    a = __reduce_max_sync(~0u, a);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHalf / 32; ++i) a = max(a, s_max[half * (kHalf / 32) + i]);
    if (page >= 0) {
      uint8_t* dst = (half ? L.c.v : L.c.k) + plane * kPage * D;
      const int e = max(need_exp(a), e_old);
      if (ht == 0) *scale = exp2_int(e);
      if (e > e_old) {                                   // the page's older rows, at the new scale
        uint4* old = reinterpret_cast<uint4*>(dst);
        for (int at = ht; at < r0 * D / 16; at += kHalf) old[at] = rescale16(old[at], e_old - e);
      }
      const float f = exp2_int(-e);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = ht + i * kHalf;
        if (at >= rows * kPerRow) continue;
        uint32_t w[2];
#pragma unroll
        for (int y = 0; y < 2; ++y)
          w[y] = static_cast<uint32_t>(float2_to_e4m3x2(x[i].at(4 * y) * f, x[i].at(4 * y + 1) * f)) |
                 (static_cast<uint32_t>(float2_to_e4m3x2(x[i].at(4 * y + 2) * f, x[i].at(4 * y + 3) * f)) << 16);
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
  }
  // Counts that go to other arrays are written at once.  Counts updated in place
  // are written by the last block to finish: every block has used the old ones by
  // then (a value that has come back cannot change, so the ticket needs no fence).
  const int add = fits ? m : 0;
  if (L.len_out != L.c.len && L.next_out != L.c.next) {
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      L.len_out[b * L.H_kv + h] = n0 + add;
      if (h == 0) L.next_out[b] = L.c.next[b] + add;
    }
    return;
  }
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = atomicAdd(L.ticket, 1) == static_cast<int>(gridDim.x * gridDim.y * gridDim.z) - 1;
  __syncthreads();
  if (!s_last) return;
  for (int s = threadIdx.x / 32; s < L.B; s += kThreads / 32) {   // a warp a sequence
    const int lane = threadIdx.x % 32;
    const int more = cache_new(L.n_new, L.n, s, L.err);
    const int grown = sequence_fits(L, s, more) ? more : 0;
    for (int i = lane; i < L.H_kv; i += 32) L.len_out[s * L.H_kv + i] = L.c.len[s * L.H_kv + i] + grown;
    if (lane == 0) L.next_out[s] = L.c.next[s] + grown;
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
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCluster = kMaxClusterBlocks;
constexpr int kSelRun = 4096;              // slots that are worth a block
constexpr int kSelKeys = 24576;            // keys that a block holds in shared memory
constexpr int kSelSmem = kSelKeys * 4 + kSelWarps * 256 * 4;

// Which slots stay.  A cluster per (sequence, head), each block over a run of its
// slots: the budget-th largest key by four passes of 8-bit counting, then the kept
// slots in order (ties: the lowest slots).  Slots are in ascending position, so
// the protected ones are among the last `recent`; only those positions are read.
// A block's keys stay in shared memory between the passes (longer runs are formed
// again in each), every warp counts into bins of its own (most keys share a few
// exponents; one addition for a warp's equal digits, found with match, was slower:
// 26.4 us against 23.4 for 8,704 slots a block), and the blocks exchange their counts through the cluster's
// distributed shared memory.
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(CacheEvictLaunch L) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  uint32_t (*s_hist)[256] = reinterpret_cast<uint32_t (*)[256]>(s_keys + kSelKeys);
  __shared__ uint32_t s_all[2][kSelCluster][256];      // the blocks' counts of a pass
  __shared__ uint2 s_counts[kSelCluster];              // the blocks' slots above and at the threshold
  __shared__ uint32_t s_sum[8], s_digit, s_left;
  __shared__ uint2 s_warp[kSelWarps];
  cg::cluster_group cluster = cg::this_cluster();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int cs = gridDim.x, rank = blockIdx.x;
  const int n = cache_len(L.src, L.H_kv, b, h, L.err);
  const int next = L.src.next[b], first_late = next - L.recent;
  const int kept = min(n, L.budget);
  int32_t* keep = L.keep + (static_cast<size_t>(b) * L.H_kv + h) * (static_cast<size_t>(L.src.max_pages) * kPage + 1);
  // whole pages per block
  const int run = ((n + kPage - 1) / kPage + cs - 1) / cs * kPage;
  const int s0 = min(n, rank * run), s1 = min(n, s0 + run);
  const bool held = run <= kSelKeys;
  auto form_key = [&](int s) {
    const int page = cache_page(L.src, b, s / kPage, L.err);
    if (page < 0) return 0u;
    const size_t at = (static_cast<size_t>(page) * L.H_kv + h) * kPage + s % kPage;
    const bool late = s >= n - L.recent && L.src.pos[at] >= first_late;
    return keep_key(L.src.mass[at], late);
  };
  auto key_of = [&](int s) { return held ? s_keys[s - s0] : form_key(s); };
  uint32_t thr = 0;
  uint32_t ties = 0;                  // slots equal to the threshold that stay
  if (n > L.budget) {
    if (held) {
      constexpr int kAtOnce = 4;        // keys whose dependent loads are in flight together
      for (int from = s0 + tid; from < s1; from += kAtOnce * kSelThreads) {
        int page[kAtOnce];
        float mass[kAtOnce];
        int pos[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int s = from + i * kSelThreads;
          page[i] = s < s1 ? L.src.table[static_cast<size_t>(b) * L.src.max_pages + s / kPage] : 0;
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int s = from + i * kSelThreads;
          const bool there = s < s1 && page[i] >= 0 && page[i] < L.src.n_pages;
          const size_t at = there ? (static_cast<size_t>(page[i]) * L.H_kv + h) * kPage + s % kPage : 0;
          mass[i] = there ? L.src.mass[at] : 0.f;
          pos[i] = there && s >= n - L.recent ? L.src.pos[at] : INT_MIN;
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int s = from + i * kSelThreads;
          if (s >= s1) break;
          const bool there = page[i] >= 0 && page[i] < L.src.n_pages;
          if (!there) atomicOr(L.err, kErrBadCache);
          s_keys[s - s0] = there ? keep_key(mass[i], s >= n - L.recent && pos[i] >= first_late) : 0u;
        }
      }
    }
    uint32_t left = L.budget;
    for (int pass = 0, shift = 24; shift >= 0; ++pass, shift -= 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s_hist[warp][lane + 32 * i] = 0;
      __syncthreads();
      for (int s = s0 + tid; s < s1; s += kSelThreads) {
        const uint32_t k = key_of(s);
        if (pass == 0 || (k >> (shift + 8)) == (thr >> (shift + 8))) atomicAdd(&s_hist[warp][(k >> shift) & 255], 1u);
      }
      if (pass == 0) asm volatile("barrier.cluster.wait;" ::: "memory");
      __syncthreads();
      uint32_t mine = 0;
      if (tid < 256) {
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) mine += s_hist[w][tid];
        for (int x = 0; x < cs; ++x) *cluster.map_shared_rank(&s_all[pass & 1][rank][tid], x) = mine;
      }
      if (cs > 1) cluster.sync(); else __syncthreads();
      // digit d = 255 - tid: the count of slots with a larger digit decides
      uint32_t here = 0, above = 0;
      if (tid < 256) {
        for (int x = 0; x < cs; ++x) here += s_all[pass & 1][x][255 - tid];
        above = here;
#pragma unroll
        for (int y = 1; y < 32; y *= 2) {
          const uint32_t v = __shfl_up_sync(~0u, above, y);
          if (lane >= y) above += v;
        }
        if (lane == 31) s_sum[warp] = above;
      }
      __syncthreads();
      if (tid < 256) {
        for (int w = 0; w < warp; ++w) above += s_sum[w];
        if (above >= left && above - here < left) {    // one thread: counts up to this digit reach `left`
          s_digit = 255 - tid;
          s_left = left - (above - here);
        }
      }
      __syncthreads();
      thr |= s_digit << shift;
      left = s_left;
    }
    ties = left;
  } else {
    asm volatile("barrier.cluster.wait;" ::: "memory");
  }
  // Ranks: slots of earlier blocks, warps and lanes.  Each warp takes a run of the
  // block's slots, so that one exchange of counts settles every rank.
  const int per_warp = ((s1 - s0 + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(s1, s0 + warp * per_warp), w1 = min(s1, w0 + per_warp);
  uint2 c = make_uint2(0, 0);         // slots above the threshold, at it
  for (int s = w0; s < w1; s += 32) {
    const uint32_t k = s + lane < w1 ? (n > L.budget ? key_of(s + lane) : 1u) : 0u;
    c.x += __popc(__ballot_sync(~0u, s + lane < w1 && k > thr));
    c.y += __popc(__ballot_sync(~0u, s + lane < w1 && n > L.budget && k == thr));
  }
  if (lane == 0) s_warp[warp] = c;
  __syncthreads();
  uint2 before = make_uint2(0, 0), total = make_uint2(0, 0);
  for (int w = 0; w < kSelWarps; ++w) {
    if (w < warp) { before.x += s_warp[w].x; before.y += s_warp[w].y; }
    total.x += s_warp[w].x;
    total.y += s_warp[w].y;
  }
  if (tid < cs) *cluster.map_shared_rank(&s_counts[rank], tid) = total;
  if (cs > 1) cluster.sync(); else __syncthreads();
  for (int x = 0; x < rank; ++x) { before.x += s_counts[x].x; before.y += s_counts[x].y; }
  for (int s = w0; s < w1; s += 32) {
    const uint32_t k = s + lane < w1 ? (n > L.budget ? key_of(s + lane) : 1u) : 0u;
    const bool over = s + lane < w1 && k > thr, tie = s + lane < w1 && n > L.budget && k == thr;
    const uint32_t ob = __ballot_sync(~0u, over), tb = __ballot_sync(~0u, tie), lanes_before = (1u << lane) - 1;
    const uint32_t tie_rank = before.y + __popc(tb & lanes_before);
    // kept slots before this one: those above the threshold and the first `ties` at it
    const uint32_t at = before.x + __popc(ob & lanes_before) + min(tie_rank, ties);
    if ((over || (tie && tie_rank < ties)) && at < static_cast<uint32_t>(kept)) keep[1 + at] = s + lane;
    before.x += __popc(ob);
    before.y += __popc(tb);
  }
  if (rank == 0 && tid == 0) {
    keep[0] = kept;
    L.dst.len[b * L.H_kv + h] = kept;
    if (h == 0) L.dst.next[b] = next;
  }
}

ClusterFits g_select_fits;

// One block per destination page and head.
template <int D>
__global__ void __launch_bounds__(kThreads, 8) cache_copy_kernel(CacheEvictLaunch L) {
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
  // All loads first: the rows' pieces and scales, and what a slot carries beside them.
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
    c[i] = __ldcs(reinterpret_cast<const uint4*>((half ? L.src.v : L.src.k) + (plane * kPage + s % kPage) * D +
                                                 (at % kPerRow) * 16));
    es[i] = scale_exp((half ? L.src.v_scale : L.src.k_scale)[plane]);
  }
  int slot_page = -1, pos = 0;
  int16_t gid = 0;
  float mass = 0.f;
  if (ht < rows) {
    const int s = keep[1 + j * kPage + ht];
    slot_page = cache_page(L.src, b, s / kPage, L.err);
    const size_t from = (static_cast<size_t>(max(slot_page, 0)) * L.H_kv + h) * kPage + s % kPage;
    if (slot_page >= 0 && half == 0) {
      pos = L.src.pos[from];
      gid = L.src.gid[from];
    } else if (slot_page >= 0) {
      mass = L.src.mass[from];
    }
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const float v = e4m3x2_to_float2(static_cast<uint16_t>(top_code(c[i]))).x * exp2_int(es[i]);
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
    if (es[i] != e) c[i] = rescale16(c[i], es[i] - e);
    __stcs(reinterpret_cast<uint4*>(dst + static_cast<size_t>(at) * 16), c[i]);
  }
  if (slot_page >= 0) {
    const size_t at = to_plane * kPage + ht;
    if (half == 0) {
      L.dst.pos[at] = pos;
      L.dst.gid[at] = gid;
    } else {
      L.dst.mass[at] = mass;
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
  // Blocks per (sequence, head): one wave, as long as each has kSelRun slots.
  const ClusterFit* fit;
  if (cudaError_t e = g_select_fits.get(L.device, reinterpret_cast<const void*>(cache_select_kernel), kSelThreads, kSelSmem, &fit))
    return e;
  int cs = 1, i = 0;
  while (cs < kSelCluster && static_cast<long long>(L.B) * L.H_kv <= fit->n[i + 1] &&
         2 * cs * kSelRun <= L.src.max_pages * kPage) {
    cs *= 2;
    ++i;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cs, L.H_kv, L.B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kSelSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, cache_select_kernel, L)) return e;
  const int cap = min(L.budget, L.src.max_pages * kPage);
  const dim3 grid((cap + kPage - 1) / kPage, L.H_kv, L.B);
  if (L.d == 128) cache_copy_kernel<128><<<grid, kThreads, 0, st>>>(L);
  else cache_copy_kernel<64><<<grid, kThreads, 0, st>>>(L);
  return cudaGetLastError();
}

}  // namespace focus
