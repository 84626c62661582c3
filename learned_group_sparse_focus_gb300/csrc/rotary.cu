// Rotation of queries and keys to their positions, alone and on the way into the paged
// 8-bit cache (contract: focus.h; the rotation's arithmetic: rotary.cuh).
//
// Both move rows once and are bound by HBM.  A token's sines and cosines serve all of its
// heads, so a block takes tokens and walks over heads.
//
// Appended keys go from the turned fp32 value to e4m3 in one rounding.  What is stored is
// what exact arithmetic would store: the fp32 value is within kUnsure of its pair's size, so
// both ends of that range are rounded, and where they give different codes (about one
// element in 10^5) or different page exponents the value is formed again in 64 bits.
// A cache then holds the same codes however its tokens came in, one by one, in a
// prompt or as a tree's path.
#include "rotary.cuh"

namespace focus {
namespace {

constexpr int kHalf = kRotThreads / 2;      // of a page's block the first half moves K, the second V
// Of |y| + |z|, for the fp32 value of a turned pair (y, z): what sine and cosine are off by (2^-22.7: the
// angle's roundings and the polynomial's), two roundings of 2^-25, and sqrt(2) for the sizes of the pair before.
constexpr float kUnsure = 0x1.8p-22f;

// ------------------------------------------------------------- rotation ---

template <typename T, int D, bool kInterleaved>
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
  rotate_rows<T, D, kInterleaved, 128>(L, b, t0, blockIdx.y * L.heads, m, L.base ? L.base[b] : 0, L.parent ? s_up : nullptr, s_turn);
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
template <typename T, int D, bool kInterleaved>
__device__ __forceinline__ void append_page(const CacheAppendRotaryLaunch& L, int b, int h, int j, int n0, int m,
                                            unsigned long long* s_turn, uint2* s_max, int* s_more, uint8_t* smem) {
  using C = PageRows<T, D>;
  const CacheAppendLaunch& A = L.a;
  const RotaryLaunch& R = L.rot;
  const int half = threadIdx.x / kHalf, ht = threadIdx.x % kHalf;
  const int lo = max(n0, j * kPage), hi = min(n0 + m, (j + 1) * kPage);
  const int r0 = lo - j * kPage, rows = hi - lo, t0 = lo - n0;
  const int k = ht % C::kDuos, row0 = ht / C::kDuos;
  const Duo duo(k, half ? 0 : R.dim, kInterleaved);
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
  fill_turns<C::kDuos>(R, s_turn);
  if (threadIdx.x == 0) *s_more = 0;
  cp_async_wait_all();
  __syncthreads();
  // A duo of a row step as floats, as it came and as it was turned.
  auto floats = [&](int i, float (&y)[16]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 f = *reinterpret_cast<const float4*>(mine + i * apart + e * C::kStep);
      y[4 * e] = f.x; y[4 * e + 1] = f.y; y[4 * e + 2] = f.z; y[4 * e + 3] = f.w;
    }
  };
  auto read = [&](int i, float (&y)[16]) {
    if constexpr (sizeof(T) == 4) {
      floats(i, y);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 u = *reinterpret_cast<const uint4*>(mine + i * apart + e * C::kStep);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          y[8 * e + 2 * x] = __uint_as_float((&u.x)[x] << 16);
          y[8 * e + 2 * x + 1] = __uint_as_float((&u.x)[x] & 0xffff0000u);
        }
      }
    }
  };
  // Turned rows, and the largest finite magnitude.
  float top = 0.f;
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    float y[16];
    read(i, y);
    if (!half) {
      if (duo.turns) {
        uint64_t c[4], s[4];
        duo_cos_sin<C::kDuos>(static_cast<uint32_t>(next) + (t0 + row0 + i * C::kRowsAtOnce), s_turn + k, R.scale, R.scale, c, s);
        turn_pairs<kInterleaved>(y, c, s);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4*>(mine + i * apart + e * C::kStep) = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
    }
    float a = 0.f, b = 0.f;                              // (fmaxf leaves NaN out)
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      a = fmaxf(a, fabsf(y[e]));
      b = fmaxf(b, fabsf(y[e + 1]));
    }
    a = fmaxf(a, b);
    if (a == INFINITY) {
      a = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) a = fmaxf(a, fabsf(y[e]) < INFINITY ? fabsf(y[e]) : 0.f);
    }
    top = fmaxf(top, a);
  }
  {
    const uint32_t fixed = __reduce_max_sync(~0u, duo.turns ? 0u : __float_as_uint(top));
    const uint32_t turned = __reduce_max_sync(~0u, duo.turns ? __float_as_uint(top) : 0u);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = make_uint2(fixed, turned);
  }
  __syncthreads();
  uint32_t fixed = 0, turned = 0;                        // largest of the elements as they came, of the turned ones
#pragma unroll
  for (int i = 0; i < kHalf / 32; ++i) {
    fixed = max(fixed, s_max[half * (kHalf / 32) + i].x);
    turned = max(turned, s_max[half * (kHalf / 32) + i].y);
  }
  auto exactly = [&](int i, int e) {                     // element e of row step i in 64 bits
    const int t = t0 + row0 + i * C::kRowsAtOnce;
    const T* row = src + static_cast<size_t>(source(t)) * D;
    const int pair = kInterleaved ? e / 2 : e % 8;
    const int first = kInterleaved ? duo.at[0] + 2 * pair : duo.at[0] + pair, other = kInterleaved ? 1 : R.dim / 2;
    const float a = static_cast<float>(row[first]), c = static_cast<float>(row[first + other]);
    return turned_exactly(a, c, (static_cast<unsigned long long>(next) + t) * s_turn[pair * C::kDuos + k], R.scale,
                          kInterleaved ? e & 1 : e >= 8);
  };
  // In exact arithmetic the largest turned one is within 2 kUnsure of `turned`.
  const float most = __uint_as_float(turned) * (1.f + 2.f * kUnsure);
  int e_new = max(need_exp(fixed), need_exp(__float_as_uint(__uint_as_float(turned) * (1.f - 2.f * kUnsure))));
  if (need_exp(__float_as_uint(most)) > e_new) {         // the same in the whole half; not in V's, where nothing turns
    const float edge = exp2_int(e_new) * 448.f;          // (infinite past fp32's range: then nothing is past it)
    if (duo.turns)
#pragma unroll 1
      for (int x = 0; x < steps * 16; ++x) {
        const float y = *reinterpret_cast<const float*>(mine + x / 16 * apart + x % 16 / 4 * C::kStep + x % 4 * 4);
        if (!(fabsf(y) >= edge * (1.f - 4.f * kUnsure) && fabsf(y) < INFINITY)) continue;
        if (fabs(exactly(x / 16, x % 16)) > edge) atomicOr(s_more, 1);
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
    uint32_t w[4];
    if (half) {
      read(i, y);
#pragma unroll
      for (int z = 0; z < 4; ++z)
        w[z] = static_cast<uint32_t>(float2_to_e4m3x2(y[4 * z] * f, y[4 * z + 1] * f)) |
               static_cast<uint32_t>(float2_to_e4m3x2(y[4 * z + 2] * f, y[4 * z + 3] * f)) << 16;
    } else {
      floats(i, y);
      // both ends of what an element may be, by its pair's size; where they differ, in 64 bits
      float u[16];
      const float unsure = kUnsure * f;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int a = kInterleaved ? 2 * x : x, b = kInterleaved ? 2 * x + 1 : x + 8;
        u[a] = u[b] = duo.turns ? (fabsf(y[a]) + fabsf(y[b])) * unsure : 0.f;
      }
      const uint64_t f2 = f2_pack(f, f), minus = f2_pack(-1.f, -1.f);
      uint32_t differ[4];                                // by byte
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        uint32_t low = 0, high = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int a = 4 * z + 2 * x;
          const uint64_t y2 = f2_pack(y[a], y[a + 1]), u2 = f2_pack(u[a], u[a + 1]);
          float v0, v1;
          f2_unpack(f2_fma(y2, f2, f2_mul(u2, minus)), v0, v1);
          low |= static_cast<uint32_t>(float2_to_e4m3x2(v0, v1)) << 16 * x;
          f2_unpack(f2_fma(y2, f2, u2), v0, v1);
          high |= static_cast<uint32_t>(float2_to_e4m3x2(v0, v1)) << 16 * x;
        }
        w[z] = low;
        differ[z] = low ^ high;
      }
      if (differ[0] | differ[1] | differ[2] | differ[3])
#pragma unroll 1
        for (int x = 0; x < 16; ++x) {
          const uint32_t word = x < 4 ? differ[0] : x < 8 ? differ[1] : x < 12 ? differ[2] : differ[3];
          if (!(word >> x % 4 * 8 & 255u)) continue;
          const uint32_t code = code_of(exactly(i, x) * exp2_int(-e)) << x % 4 * 8, rest = ~(255u << x % 4 * 8);
#pragma unroll
          for (int z = 0; z < 4; ++z)
            if (z == x / 4) w[z] = (w[z] & rest) | code;
        }
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

// Grid x: blocks of pages, one per touched page and head, and those of query rows, spread evenly
// among each other: the former are bound by instructions, the latter by HBM.
template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads, 3) cache_append_rotary_kernel(CacheAppendRotaryLaunch L) {
  __shared__ unsigned long long s_turn[D / 2];
  __shared__ uint2 s_max[kRotThreads / 32];
  __shared__ int s_more;
  extern __shared__ __align__(16) uint8_t smem[];
  const CacheAppendLaunch& A = L.a;
  const int b = blockIdx.z;
  const int m = cache_new(A.n_new, A.n, b, A.err);
  const bool fits = sequence_fits(A, b, m);
  if (!fits && threadIdx.x == 0) atomicOr(A.err, kErrBadCache);
  const unsigned long long of_pages = static_cast<unsigned long long>(L.touched) * A.H_kv;
  const uint32_t before = static_cast<uint32_t>(blockIdx.x * of_pages / gridDim.x);      // blocks of pages before this one
  const bool is_page = static_cast<uint32_t>((blockIdx.x + 1ull) * of_pages / gridDim.x) > before;
  int h = 0, n0 = 0;
  if (is_page) {
    h = before / L.touched;
    n0 = A.c.len[b * A.H_kv + h];
    const int j = n0 / kPage + before % L.touched;
    if (fits && max(n0, j * kPage) < min(n0 + m, (j + 1) * kPage)) append_page<T, D, kInterleaved>(L, b, h, j, n0, m, s_turn, s_max, &s_more, smem);
  } else if (fits) {
    const int x = blockIdx.x - before, chunks = (A.n + L.rot.tokens - 1) / L.rot.tokens;
    const int t0 = x % chunks * L.rot.tokens;
    if (t0 < m) rotate_rows<T, D, kInterleaved, 64>(L.rot, b, t0, x / chunks * L.rot.heads, m, A.c.next[b], nullptr, s_turn);
  }
  append_counts(A, b, h, n0, fits ? m : 0, is_page && before % L.touched == 0,
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
template <typename T, int D, bool kInterleaved>
std::atomic<bool> g_ready[kMaxDevices];

template <typename T, int D, bool kInterleaved>
cudaError_t launch_append(const CacheAppendRotaryLaunch& L, dim3 grid, cudaStream_t st) {
  constexpr int kSmem = PageRows<T, D>::kBytes;
  const auto kernel = cache_append_rotary_kernel<T, D, kInterleaved>;
  std::atomic<bool>& ready = g_ready<T, D, kInterleaved>[L.device];
  if (!ready.load(std::memory_order_acquire)) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) return e;
    ready.store(true, std::memory_order_release);
  }
  kernel<<<grid, kRotThreads, kSmem, st>>>(L);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_append(const CacheAppendRotaryLaunch& L, dim3 grid, cudaStream_t st) {
  return L.rot.interleaved ? launch_append<T, D, true>(L, grid, st) : launch_append<T, D, false>(L, grid, st);
}

template <typename T, int D>
cudaError_t launch_rows(const RotaryLaunch& L, dim3 grid, cudaStream_t st) {
  if (L.interleaved) rotary_kernel<T, D, true><<<grid, kRotThreads, 0, st>>>(L);
  else rotary_kernel<T, D, false><<<grid, kRotThreads, 0, st>>>(L);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(RotaryLaunch L, int d, int dtype, cudaStream_t st) {
  split_rows(&L, d);
  const dim3 grid((L.n + L.tokens - 1) / L.tokens, (L.Hq + L.Hk + L.heads - 1) / L.heads, L.B);
  if (dtype == FOCUS_BF16) return d == 128 ? launch_rows<__nv_bfloat16, 128>(L, grid, st) : launch_rows<__nv_bfloat16, 64>(L, grid, st);
  return d == 128 ? launch_rows<float, 128>(L, grid, st) : launch_rows<float, 64>(L, grid, st);
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
