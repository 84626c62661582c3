// Rotation of queries and keys to their positions, alone and on the way into the paged
// 8-bit cache (contract: focus.h; the rotation's arithmetic: rotary.cuh).
//
// Both move rows once and are bound by HBM.  A token's sines and cosines serve all of its
// heads, so a block takes tokens and walks over heads.
//
// Appended keys go from the turned fp32 value to e4m3 in one rounding.  What is stored is
// what exact arithmetic would store: the fp32 value is within 2^-20 of its pair's size, so
// both ends of that range are rounded, and where they give different codes (about one
// element in 10^5) or different page exponents the value is formed again in 64 bits.
// A cache then holds the same codes however its tokens came in, one by one, in a
// prompt or as a tree's path.
#include "rotary.cuh"

namespace focus {
namespace {

constexpr int kHalf = kRotThreads / 2;      // of a page's block the first half moves K, the second V
constexpr float kUnsure = 0x1p-20f;         // of |a| + |b|, for the fp32 value of a turned pair (a, b)

// ------------------------------------------------------------- rotation ---

template <typename T, int D>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(RotaryLaunch L) {
  __shared__ unsigned long long s_turn[D / 2];
  __shared__ unsigned long long s_line[kMaxNodes];
  __shared__ int s_up[kMaxNodes];
  const int b = blockIdx.z;
  const int m = cache_new(L.n_new, L.n, b, L.err);
  const int t0 = blockIdx.x * L.tokens;
  if (t0 >= m) return;
  if (L.parent) {
    if (threadIdx.x < 32) {
      tree_lines(L.parent + static_cast<size_t>(b) * L.n, m, s_line, s_up, L.err);
#pragma unroll
      for (int i = 0; i < 2; ++i) s_up[threadIdx.x + 32 * i] = __popcll(s_line[threadIdx.x + 32 * i]) - 1;
    }
    __syncthreads();
  }
  rotate_rows<T, D>(L, b, t0, blockIdx.y * L.heads, m, L.base ? L.base[b] : 0, L.parent ? s_up : nullptr, s_turn);
}

// --------------------------------------------------------------- append ---

// A turned pair in 64 bits: element hi (0, 1) of (a, b) at a phase in 2^-64 turns.  Taylor
// polynomials of degree 15 and 16 on an eighth of a turn, as in cos_sin (the next terms are below
// 2^-54 and 2^-58).  A call: it is needed for few elements, and its code would crowd out the rest.
__device__ __noinline__ double turned_exactly(float a, float b, unsigned long long phase, float scale, bool hi) {
  const uint32_t quarter = static_cast<uint32_t>((phase + (1ull << 61)) >> 62);
  const long long rest = static_cast<long long>(phase - (static_cast<unsigned long long>(quarter) << 62));
  const double x = static_cast<double>(rest) * (6.283185307179586477 * 0x1p-64), z = x * x;
  double s = -1. / 1307674368000., c = 1. / 20922789888000.;     // -1 / 15!, 1 / 16!
  s = fma(s, z, 1. / 6227020800.);
  c = fma(c, z, -1. / 87178291200.);
  s = fma(s, z, -1. / 39916800.);
  c = fma(c, z, 1. / 479001600.);
  s = fma(s, z, 1. / 362880.);
  c = fma(c, z, -1. / 3628800.);
  s = fma(s, z, -1. / 5040.);
  c = fma(c, z, 1. / 40320.);
  s = fma(s, z, 1. / 120.);
  c = fma(c, z, -1. / 720.);
  s = fma(s, z, -1. / 6.);
  c = fma(c, z, 1. / 24.);
  c = fma(c, z, -0.5);
  s = fma(x * z, s, x);
  c = fma(c, z, 1.);
  double cq = quarter & 1 ? s : c, sq = quarter & 1 ? c : s;
  if (quarter == 1 || quarter == 2) cq = -cq;
  if (quarter >= 2) sq = -sq;
  const double u = a, v = b;
  return (hi ? u * sq + v * cq : u * cq - v * sq) * scale;
}

// e4m3 code of a double, rounded once: to a float by truncation with the lost bits in its
// last one, which the rounding to e4m3 reads like any bits below the half.
__device__ __forceinline__ uint32_t code_of(double y) {
  float f = __double2float_rz(y);
  if (static_cast<double>(f) != y) f = __uint_as_float(__float_as_uint(f) | 1u);
  return float2_to_e4m3x2(f, 0.f) & 0xffu;
}

// A page's rows in shared memory: a thread's duos, row step after row step, in 16-byte
// pieces that lie a thread apart.  K's are turned in place (fp32), V's stay as they are.
template <typename T, int D>
struct PageRows {
  static constexpr int kDuos = D / 16, kRowsAtOnce = kHalf / kDuos, kSteps = kPage / kRowsAtOnce;
  static constexpr int kRaw = sizeof(T);                 // 16-byte pieces of a duo as it comes: 2 or 4
  static constexpr int kStep = kHalf * 16;               // bytes of one piece of every thread
  static constexpr int kBytes = kSteps * (4 + kRaw) * kStep;
};

// One page of one head: as cache_append_kernel, with a thread on duos.
template <typename T, int D>
__device__ __forceinline__ void append_page(const CacheAppendRotaryLaunch& L, int b, int h, int j, int n0, int m,
                                            unsigned long long* s_turn, uint32_t (*s_max)[2], int* s_more, uint8_t* smem) {
  using C = PageRows<T, D>;
  const CacheAppendLaunch& A = L.a;
  const RotaryLaunch& R = L.rot;
  const int half = threadIdx.x / kHalf, ht = threadIdx.x % kHalf;
  const int lo = max(n0, j * kPage), hi = min(n0 + m, (j + 1) * kPage);
  const int r0 = lo - j * kPage, rows = hi - lo, t0 = lo - n0;
  const int k = ht % C::kDuos, row0 = ht / C::kDuos;
  const Duo duo(k, half ? 0 : R.dim, R.interleaved);
  const int next = A.c.next[b];
  // the source row of a token
  auto source = [&](int t) {
    if (!L.rows) return t;
    const int r = L.rows[static_cast<size_t>(b) * A.n + t];
    if (r >= 0 && r < A.n) return r;
    atomicOr(A.err, kErrBadTree);
    return r < 0 ? 0 : A.n - 1;
  };
  const T* src = static_cast<const T*>(half ? A.V : A.K) + (static_cast<size_t>(b) * A.H_kv + h) * A.n * D;
  uint8_t* const mine = smem + (half ? C::kSteps * 4 * C::kStep : 0) + ht * 16;
  const int apart = (half ? C::kRaw : 4) * C::kStep;     // from a row step to the next
  const int steps = row0 < rows ? (rows - row0 + C::kRowsAtOnce - 1) / C::kRowsAtOnce : 0;
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    const T* row = src + static_cast<size_t>(source(t0 + row0 + i * C::kRowsAtOnce)) * D;
#pragma unroll
    for (int e = 0; e < C::kRaw; ++e)
      cp_async_16(mine + i * apart + e * C::kStep, row + duo.at[e / (C::kRaw / 2)] + e % (C::kRaw / 2) * (16 / static_cast<int>(sizeof(T))), 16);
  }
  const int page = cache_page(A.c, b, j, A.err);
  const size_t plane = static_cast<size_t>(max(page, 0)) * A.H_kv + h;
  float* scale = (half ? A.c.v_scale : A.c.k_scale) + plane;
  const int e_old = r0 > 0 && page >= 0 ? scale_exp(*scale) : kMinExp;
  if (threadIdx.x < R.dim / 2) s_turn[threadIdx.x] = turn_of(R.inv_freq[threadIdx.x]);
  if (threadIdx.x == 0) *s_more = 0;
  cp_async_wait_all();
  __syncthreads();
  // A duo of a row step as floats; y: K's turned ones.
  auto read = [&](int i, bool turned, float (&y)[16]) {
    const uint8_t* at = mine + i * apart;
    if (sizeof(T) == 4 || turned) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 f = *reinterpret_cast<const float4*>(at + (sizeof(T) == 4 || turned ? e : 0) * C::kStep);
        y[4 * e] = f.x; y[4 * e + 1] = f.y; y[4 * e + 2] = f.z; y[4 * e + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 u = *reinterpret_cast<const uint4*>(at + e * C::kStep);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          y[8 * e + 2 * x] = __uint_as_float((&u.x)[x] << 16);
          y[8 * e + 2 * x + 1] = __uint_as_float((&u.x)[x] & 0xffff0000u);
        }
      }
    }
  };
  // how far an element may be from exact arithmetic, by its pair's size
  auto unsure = [&](const float (&y)[16], int e) {
    if (!duo.turns) return 0.f;
    const float other = R.interleaved ? y[e ^ 1] : y[e ^ 8];
    return (fabsf(y[e]) + fabsf(other)) * kUnsure;
  };
  // Turned rows, their largest finite magnitude, and the most that it may be in exact arithmetic.
  uint32_t top[2] = {0, 0};
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    float y[16];
    read(i, false, y);
    if (duo.turns) {
      float c[8], s[8];
      const unsigned long long x = static_cast<unsigned long long>(next) + (t0 + row0 + i * C::kRowsAtOnce);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cos_sin(x * s_turn[k * 8 + e], c[e], s[e]);
        c[e] *= R.scale;
        s[e] *= R.scale;
      }
      if (R.interleaved) turn_pairs<true>(y, c, s);
      else turn_pairs<false>(y, c, s);
    }
    if (!half)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4*>(mine + i * apart + e * C::kStep) = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float a = fabsf(y[e]);
      if (!(a < INFINITY)) continue;
      const float u = unsure(y, e);
      top[0] = max(top[0], __float_as_uint(fmaxf(a - u, 0.f)));
      top[1] = max(top[1], __float_as_uint(a + u < INFINITY ? a + u : a));
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) top[x] = __reduce_max_sync(~0u, top[x]);
  if ((threadIdx.x & 31) == 0) {
    s_max[threadIdx.x / 32][0] = top[0];
    s_max[threadIdx.x / 32][1] = top[1];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHalf / 32; ++i) {
    top[0] = max(top[0], s_max[half * (kHalf / 32) + i][0]);
    top[1] = max(top[1], s_max[half * (kHalf / 32) + i][1]);
  }
  auto exactly = [&](int i, int e) {                     // element e of row step i in 64 bits
    const int t = t0 + row0 + i * C::kRowsAtOnce;
    const T* row = src + static_cast<size_t>(source(t)) * D;
    const int pair = R.interleaved ? e / 2 : e % 8;
    const int first = R.interleaved ? duo.at[0] + 2 * pair : duo.at[0] + pair, other = R.interleaved ? 1 : R.dim / 2;
    const float a = static_cast<float>(row[first]), c = static_cast<float>(row[first + other]);
    return turned_exactly(a, c, (static_cast<unsigned long long>(next) + t) * s_turn[k * 8 + pair], R.scale,
                          R.interleaved ? e & 1 : e >= 8);
  };
  int e_new = need_exp(top[0]);
  if (!half && need_exp(top[1]) != e_new) {              // the same in the whole half
    const double edge = static_cast<double>(exp2_int(e_new)) * 448.0;
    if (duo.turns)
#pragma unroll 1
      for (int x = 0; x < steps * 16; ++x) {
        const double v = fabs(exactly(x / 16, x % 16));
        if (v > edge && v < INFINITY && v <= static_cast<double>(__uint_as_float(top[1]))) atomicOr(s_more, 1);
      }
    named_barrier(1, kHalf);
    e_new += *s_more;
  }
  uint8_t* dst = (half ? A.c.v : A.c.k) + plane * kPage * D;
  const int e = max(e_new, e_old);
  if (page >= 0) {
    if (ht == 0) *scale = exp2_int(e);
    if (e > e_old) {                                     // the page's older rows, at the new scale
      uint4* old = reinterpret_cast<uint4*>(dst);
#pragma unroll 1
      for (int at = ht; at < r0 * D / 16; at += kHalf) old[at] = rescale16(old[at], e_old - e);
    }
  }
  // Rows that K_out shares with K are read in 64 bits, where that is needed, before they are written.
  const float f = exp2_int(-e);
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    const int r = row0 + i * C::kRowsAtOnce;
    float y[16];
    read(i, !half, y);
    uint32_t w[4], differ = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      uint32_t code;
      if (duo.turns) {
        const float u0 = unsure(y, 2 * x), u1 = unsure(y, 2 * x + 1);
        code = float2_to_e4m3x2((y[2 * x] - u0) * f, (y[2 * x + 1] - u1) * f);
        differ |= code != float2_to_e4m3x2((y[2 * x] + u0) * f, (y[2 * x + 1] + u1) * f) ? 1u << x : 0u;
      } else {
        code = float2_to_e4m3x2(y[2 * x] * f, y[2 * x + 1] * f);
      }
      if (x & 1) w[x / 2] |= code << 16;
      else w[x / 2] = code;
    }
#pragma unroll 1
    for (; differ; differ &= differ - 1) {
      const int x = __ffs(differ) - 1;
      const double down = exp2_int(-e);
      const uint32_t code = code_of(exactly(i, 2 * x) * down) | code_of(exactly(i, 2 * x + 1) * down) << 8;
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (z == x / 2) w[z] = x & 1 ? (w[z] & 0xffffu) | code << 16 : (w[z] & 0xffff0000u) | code;
    }
    if (page >= 0) {
      uint8_t* to = dst + static_cast<size_t>(r0 + r) * D;
      *reinterpret_cast<uint2*>(to + duo.at[0]) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(to + duo.at[1]) = make_uint2(w[2], w[3]);
    }
    if (!half && R.K_out) {
      T* out = static_cast<T*>(R.K_out) + ((static_cast<size_t>(b) * A.H_kv + h) * A.n + t0 + r) * D;
      store8(out + duo.at[0], y);
      store8(out + duo.at[1], y + 8);
    }
  }
  if (page >= 0 && ht < rows) {
    const size_t at = plane * kPage + r0 + ht;
    if (half == 0) {
      int g = A.gid[(static_cast<size_t>(b) * A.A + (A.A == 1 ? 0 : h)) * A.n + source(t0 + ht)];
      if (g < 0 || g >= A.K_groups) {
        atomicOr(A.err, kErrBadGroup);
        g = g < 0 ? 0 : A.K_groups - 1;
      }
      A.c.pos[at] = next + t0 + ht;
      A.c.gid[at] = static_cast<int16_t>(g);
    } else if (A.c.mass) {
      A.c.mass[at] = 0.f;
    }
  }
}

// Grid x: first the blocks of pages, one per touched page and head, then those of query rows.
template <typename T, int D>
__global__ void __launch_bounds__(kRotThreads, 3) cache_append_rotary_kernel(CacheAppendRotaryLaunch L) {
  __shared__ unsigned long long s_turn[D / 2];
  __shared__ uint32_t s_max[kRotThreads / 32][2];
  __shared__ int s_more;
  extern __shared__ __align__(16) uint8_t smem[];
  const CacheAppendLaunch& A = L.a;
  const int b = blockIdx.z;
  const int m = cache_new(A.n_new, A.n, b, A.err);
  const bool fits = sequence_fits(A, b, m);
  if (!fits && threadIdx.x == 0) atomicOr(A.err, kErrBadCache);
  const int of_pages = L.touched * A.H_kv;
  int h = 0, n0 = 0;
  if (static_cast<int>(blockIdx.x) < of_pages) {
    h = blockIdx.x / L.touched;
    n0 = A.c.len[b * A.H_kv + h];
    const int j = n0 / kPage + blockIdx.x % L.touched;
    if (fits && max(n0, j * kPage) < min(n0 + m, (j + 1) * kPage)) append_page<T, D>(L, b, h, j, n0, m, s_turn, s_max, &s_more, smem);
  } else if (fits) {
    const int x = blockIdx.x - of_pages, chunks = (A.n + L.rot.tokens - 1) / L.rot.tokens;
    const int t0 = x % chunks * L.rot.tokens;
    if (t0 < m) rotate_rows<T, D>(L.rot, b, t0, x / chunks * L.rot.heads, m, A.c.next[b], nullptr, s_turn);
  }
  append_counts(A, b, h, n0, fits ? m : 0, static_cast<int>(blockIdx.x) < of_pages && blockIdx.x % L.touched == 0,
                gridDim.x * gridDim.y * gridDim.z);
}

// Tokens a block and heads it walks over: as many tokens as its threads hold (what a
// head's rows in memory are long), all heads, unless the blocks are too few for the SMs.
void split_rows(RotaryLaunch* L, int d) {
  const int slots = kRotThreads / (d / 16), all = L->Hq + L->Hk;
  L->tokens = 1;
  while (L->tokens < slots && L->tokens < L->n) L->tokens *= 2;
  L->heads = all;
  const long long blocks = static_cast<long long>(L->B) * ((L->n + L->tokens - 1) / L->tokens);
  const int least = slots / L->tokens;
  while (L->heads > least && blocks * ((all + L->heads - 1) / L->heads) < kFillBlocks) L->heads = (L->heads + 1) / 2;
}

// Devices on which the kernel's shared memory is set up.
template <typename T, int D>
std::atomic<bool> g_ready[kMaxDevices];

template <typename T, int D>
cudaError_t launch_append(const CacheAppendRotaryLaunch& L, dim3 grid, cudaStream_t st) {
  constexpr int kSmem = PageRows<T, D>::kBytes;
  const void* kernel = reinterpret_cast<const void*>(cache_append_rotary_kernel<T, D>);
  if (!g_ready<T, D>[L.device].load(std::memory_order_acquire)) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) return e;
    g_ready<T, D>[L.device].store(true, std::memory_order_release);
  }
  cache_append_rotary_kernel<T, D><<<grid, kRotThreads, kSmem, st>>>(L);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(RotaryLaunch L, int d, int dtype, cudaStream_t st) {
  split_rows(&L, d);
  const dim3 grid((L.n + L.tokens - 1) / L.tokens, (L.Hq + L.Hk + L.heads - 1) / L.heads, L.B);
  if (dtype == FOCUS_BF16) {
    if (d == 128) rotary_kernel<__nv_bfloat16, 128><<<grid, kRotThreads, 0, st>>>(L);
    else rotary_kernel<__nv_bfloat16, 64><<<grid, kRotThreads, 0, st>>>(L);
  } else {
    if (d == 128) rotary_kernel<float, 128><<<grid, kRotThreads, 0, st>>>(L);
    else rotary_kernel<float, 64><<<grid, kRotThreads, 0, st>>>(L);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_append_rotary(CacheAppendRotaryLaunch L, int dtype, cudaStream_t st) {
  L.touched = (L.a.n + kPage - 2) / kPage + 1;           // pages that n new slots from anywhere in a page touch
  unsigned long long blocks = static_cast<unsigned long long>(L.touched) * L.a.H_kv;
  if (L.rot.Hq) {
    split_rows(&L.rot, L.a.d);
    blocks += static_cast<unsigned long long>((L.a.n + L.rot.tokens - 1) / L.rot.tokens) *
              ((L.rot.Hq + L.rot.heads - 1) / L.rot.heads);
  }
  const dim3 grid(static_cast<unsigned>(blocks), 1, L.a.B);
  if (dtype == FOCUS_BF16) return L.a.d == 128 ? launch_append<__nv_bfloat16, 128>(L, grid, st) : launch_append<__nv_bfloat16, 64>(L, grid, st);
  return L.a.d == 128 ? launch_append<float, 128>(L, grid, st) : launch_append<float, 64>(L, grid, st);
}

}  // namespace focus
