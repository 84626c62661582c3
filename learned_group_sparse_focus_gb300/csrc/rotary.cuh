// Position rotation of query and key rows (contract: focus.h).
//
// A pair of elements turns by x * f, x the row's position and f the pair's frequency.
// fp32 loses that angle at far positions (x * f mod 2 pi is off by 2^-24 x f), so it
// is kept as a fraction of a turn in 64-bit fixed point: x * t modulo 2^64, with
// t = f / (2 pi) times 2^64, wraps by itself and is off by at most 2^-33 turns for any
// 32-bit x.  The turn is taken to the nearest quarter, so sine and cosine see at most
// an eighth of a turn, held to 2^-24 of itself, and are off by less than 2^-23.
//
// A thread turns a "duo" of two 8-element pieces of a row: elements k * 8 + e and
// r / 2 + k * 8 + e, or, for neighbouring pairs, the 16 from k * 16 on; both use the
// frequencies k * 8 ... k * 8 + 7, so sines and cosines stay in registers from head
// to head.
#pragma once

#include "append.cuh"
#include "tree.cuh"

namespace focus {

constexpr int kRotThreads = kAppendThreads;

// t of a frequency: its 24 bits times 1 / (2 pi) to 128, shifted into place; the bits above
// are whole turns.  A double would be off by 2^-53 of f / (2 pi), 2^-22 of it at position 2^31.
__device__ __forceinline__ unsigned long long turn_of(float inv_freq) {
  const unsigned long long hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;       // 2^128 / (2 pi)
  const uint32_t u = __float_as_uint(inv_freq), exponent = u >> 23 & 255u;
  const unsigned long long m = (u & 0x7fffffu) | (exponent ? 0x800000u : 0u);
  const unsigned long long p0 = m * lo, carry = __umul64hi(m, lo), p1 = m * hi + carry;
  const unsigned long long p2 = __umul64hi(m, hi) + (p1 < carry ? 1u : 0u);
  const int shift = 64 + 150 - static_cast<int>(exponent ? exponent : 1u);   // of the 152-bit product, down
  unsigned long long t = 0;                                        // infinities, NaN and |f| >= 2^87 among them
  if (shift >= 128 && shift < 192) t = p2 >> (shift - 128);
  else if (shift >= 64 && shift < 128) t = shift == 64 ? p1 : p1 >> (shift - 64) | p2 << (128 - shift);
  else if (shift >= 0 && shift < 64) t = shift == 0 ? p0 : p0 >> shift | p1 << (64 - shift);
  return u >> 31 ? 0ull - t : t;
}

// Cosine and sine of a phase in 2^-64 turns: Taylor polynomials of degree 10 and 9 on an
// eighth of a turn (the next terms are below 2^-32 and 2^-29), evaluated in fp32.
__device__ __forceinline__ void cos_sin(unsigned long long phase, float& c, float& s) {
  const uint32_t quarter = static_cast<uint32_t>((phase + (1ull << 61)) >> 62);
  const long long rest = static_cast<long long>(phase - (static_cast<unsigned long long>(quarter) << 62));   // at most an eighth
  const float x = static_cast<float>(static_cast<int>(rest >> 30)) * (3.14159265358979f * 0x1p-33f);   // bits 61 ... 30: |rest| <= 2^61
  const float z = x * x;
  const float a = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f), -0.16666667f), x);
  const float b = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f), 4.1666667e-2f), -0.5f), 1.f);
  c = quarter & 1 ? a : b;
  s = quarter & 1 ? b : a;
  c = __uint_as_float(__float_as_uint(c) ^ ((quarter + 1) << 30 & 0x80000000u));   // negative in quarters 1 and 2
  s = __uint_as_float(__float_as_uint(s) ^ (quarter << 30 & 0x80000000u));         // in 2 and 3
}

// Pieces of duo k of a row of D elements of which the first dim are turned.
struct Duo {
  int at[2];        // first element of each piece
  bool turns;
  __device__ __forceinline__ Duo(int k, int dim, bool interleaved) {
    turns = k * 16 < dim;
    const bool apart = turns && !interleaved;
    at[0] = apart ? k * 8 : k * 16;
    at[1] = apart ? dim / 2 + k * 8 : k * 16 + 8;
  }
};

// Pair e of a duo's 16 elements y: places of its two elements.
__device__ __forceinline__ constexpr int pair_lo(int e, bool interleaved) { return interleaved ? 2 * e : e; }
__device__ __forceinline__ constexpr int pair_hi(int e, bool interleaved) { return interleaved ? 2 * e + 1 : 8 + e; }

template <bool kInterleaved>
__device__ __forceinline__ void turn_pairs(float (&y)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = y[pair_lo(e, kInterleaved)], b = y[pair_hi(e, kInterleaved)];
    y[pair_lo(e, kInterleaved)] = fmaf(-b, s[e], a * c[e]);
    y[pair_hi(e, kInterleaved)] = fmaf(b, c[e], a * s[e]);
  }
}

__device__ __forceinline__ void store8(float* p, const float* y) {
  reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* y) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                            pack_bf16x2(y[6], y[7]));
}

// Rows of a block's tokens and heads: `tokens` tokens (a power of two) of `heads` heads.
// Head g < L.H is a query head, the others are key heads.
template <typename T, int D>
__device__ __forceinline__ void rotate_rows(const RotaryLaunch& L, int b, int t0, int head0, int valid,
                                            long long first, const int* depth, unsigned long long* s_turn) {
  constexpr int kDuos = D / 16, kSlots = kRotThreads / kDuos, kAtOnce = sizeof(T) == 2 ? 4 : 2;
  if (threadIdx.x < L.dim / 2) s_turn[threadIdx.x] = turn_of(L.inv_freq[threadIdx.x]);
  __syncthreads();
  const int k = threadIdx.x % kDuos, slot = threadIdx.x / kDuos;
  const int t = t0 + slot % L.tokens, across = kSlots / L.tokens;
  if (t >= valid) return;
  const Duo duo(k, L.dim, L.interleaved);
  float c[8], s[8];
  if (duo.turns) {
    const long long x = first + (depth ? depth[t] : t);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cos_sin(static_cast<unsigned long long>(x) * s_turn[k * 8 + e], c[e], s[e]);
      c[e] *= L.scale;
      s[e] *= L.transpose ? -L.scale : L.scale;
    }
  }
  const int end = min(head0 + L.heads, L.Hq + L.Hk);
  for (int g0 = head0 + slot / L.tokens; g0 < end; g0 += across * kAtOnce) {
    Piece<T> p[kAtOnce][2];
    const T* from[kAtOnce];
    T* to[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int g = g0 + i * across;
      if (g >= end) break;
      const bool q = g < L.Hq;
      const size_t row = ((static_cast<size_t>(b) * (q ? L.Hq : L.Hk) + (q ? g : g - L.Hq)) * L.n + t) * D;
      from[i] = static_cast<const T*>(q ? L.Q : L.K) + row;
      to[i] = static_cast<T*>(q ? L.Q_out : L.K_out) + row;
      p[i][0].load(from[i] + duo.at[0]);
      p[i][1].load(from[i] + duo.at[1]);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (g0 + i * across >= end) break;
      if (!duo.turns) {                                  // as they are, to the last bit
        if (from[i] != to[i]) {
          p[i][0].store(to[i] + duo.at[0]);
          p[i][1].store(to[i] + duo.at[1]);
        }
        continue;
      }
      float y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = p[i][e / 8].at(e % 8);
      if (L.interleaved) turn_pairs<true>(y, c, s);
      else turn_pairs<false>(y, c, s);
      store8(to[i] + duo.at[0], y);
      store8(to[i] + duo.at[1], y + 8);
    }
  }
}

}  // namespace focus
