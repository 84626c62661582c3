// Focus attention of new tokens over the paged 8-bit cache (contract: focus.h).
//
// With few query rows the keys are read once and barely reused: a kept key
// costs 2 d bytes and 4 d FLOP a query row, so the bound is HBM, and for a
// single sequence the latency of one dependent chain (table, group ids, rows).
//
// Split: a cluster of blocks shares one (sequence, key/value head); pages go
// round over its blocks and their warps.  Each warp works alone from the scan to
// its partial result: it reads its pages' group ids (and, among the last
// w + n_new slots, positions: slots are in ascending position, so no earlier
// slot can lie in a window), appends the kept slots to a list in shared memory,
// and gathers their rows in tiles of 16 keys with cp.async, kStages tiles ahead.
// Only kept rows are read.
//
// Products run on mma.m16n8k16 with the keys on the 16 side and the query rows
// (tokens x query heads of the head) on the 8 side:
//   S^T = K Q^T:    thread (g, c) = (lane / 4, lane % 4) holds row g of the key
//                   fragment.  The sum over d may run in any order, so the thread
//                   takes 16 consecutive bytes of its row and Q is laid out to
//                   match: no transposition, one 16-byte load per 16 codes.
//   O^T += V^T P^T: two keys' bytes of one column are zipped with one byte
//                   permute into the pairs that the fragment wants; P^T comes
//                   from S^T by an 8x8 register transpose.
// Codes become f16 exactly.  Queries are scaled by a power of two per row to
// below 2^15 and held in one f16 (bf16 tensors: 8 bits fit 11) or two (fp32
// tensors, 22 bits).  Accumulation is fp32.
//
// Softmax: with v = code * 2^e per page, the running maximum is taken over
// t_j = s_j + e_j (log2), so the f16 weights 2^(t_j - ref) multiply raw codes and
// stay in range for pages of any scale; the row sum adds 2^(t_j - ref) 2^-e_j in
// fp32.  ref lies 7 below the maximum when it is set and is moved only when a
// weight would pass 2^15, so f16's subnormals begin 2^-21 below the largest one.
//
// The warps' partials are joined in shared memory, the blocks' through the
// cluster's distributed shared memory, each block writing a part of the rows.
// With accumulate, logits of the kept slots go to scratch (4 bytes a row and
// key, against 2 d bytes of key and value) and are turned into weights after
// the join, by the warp that wrote them: no atomics, a fixed order.
#include <cooperative_groups.h>
#include <type_traits>

#include "cache.cuh"

namespace cg = cooperative_groups;

namespace focus {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = 16;            // keys of a tile
constexpr int kStages = 2;           // tiles in flight per warp
constexpr int kFar = INT_MIN;        // list position of a slot outside every window
constexpr int kListBytes = 4096;     // a warp's list of kept slots

template <typename T, int D, int NT, bool kMulti>
struct Cfg {
  static constexpr int kBatch = kMulti ? 2 : 4;                           // pages scanned at a time
  static constexpr int kList = kListBytes / (kMulti ? 16 : 8);            // list entries
  static_assert(kList >= kBatch * kPage + (kStages + 2) * kKeys && (kList & (kList - 1)) == 0, "list too short");
  static constexpr int kParts = std::is_same<T, float>::value ? 2 : 1;   // f16 parts of q and of P
  static constexpr int kRows = 8 * NT;
  static constexpr int kStageBytes = 2 * kKeys * D;                       // K rows, then V rows
  static constexpr int kRing = kStages * kStageBytes > kRows * D * 4 ? kStages * kStageBytes : kRows * D * 4;
  static constexpr int kWarpBytes = kRing + kListBytes;
  static constexpr int kSmem = kWarps * kWarpBytes;
  static constexpr int kSteps = D / 16;                                   // MMA steps over d
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

__device__ __forceinline__ void load4(const float* p, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* f) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(u.x << 16); f[1] = __uint_as_float(u.x & 0xffff0000u);
  f[2] = __uint_as_float(u.y << 16); f[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

// A warp's walk over its pages.  Table entries and scales are fetched for 32 pages at a time, one page a lane;
// group ids and positions kBatch pages at a time, one batch ahead of their use.
template <int kBatch>
struct Scan {
  int first, step, pages, n, near_from;        // the warp's pages: first, first + step, ...
  int k;                                       // ordinal of the batch in registers
  int lane_page, lane_exp;                     // per lane: page and exponents of 32 pages
  int page[kBatch], exps[kBatch];
  uint32_t ids[kBatch];
  int2 pos[kBatch];

  __device__ __forceinline__ void fetch(const CacheAttnLaunch& L, int b, int h, int lane) {
    if ((k & 31) == 0) {
      const int j = first + (k + lane) * step;
      lane_page = -1;
      lane_exp = 0;
      if (j < pages) lane_page = cache_page(L.c, b, j, L.err);
      if (lane_page >= 0) {
        const size_t plane = static_cast<size_t>(lane_page) * L.H_kv + h;
        lane_exp = (scale_exp(L.c.k_scale[plane]) & 0xffff) | (scale_exp(L.c.v_scale[plane]) << 16);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      page[i] = __shfl_sync(~0u, lane_page, (k + i) & 31);
      exps[i] = __shfl_sync(~0u, lane_exp, (k + i) & 31);
      ids[i] = 0;
      pos[i] = make_int2(kFar, kFar);
      if (page[i] >= 0) {
        const int j = first + (k + i) * step;
        const size_t at = (static_cast<size_t>(page[i]) * L.H_kv + h) * kPage + 2 * lane;
        ids[i] = *reinterpret_cast<const uint32_t*>(L.c.gid + at);
        if ((j + 1) * kPage > near_from) pos[i] = *reinterpret_cast<const int2*>(L.c.pos + at);
      }
    }
  }

  __device__ __forceinline__ bool done() const { return first + k * step >= pages; }
};

template <typename T, int D, int NT, bool kMulti>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) cache_attn_kernel(CacheAttnLaunch L) {
  using C = Cfg<T, D, NT, kMulti>;
  constexpr int kBatch = C::kBatch, kList = C::kList;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];
  __shared__ float s_M[C::kRows], s_L[C::kRows];       // the block's reference and sum per row
  __shared__ float s_lse[C::kRows];                    // log2 sum-exp of the whole row
  __shared__ int s_gid[C::kRows];                      // group id of each token of the row block
  const int h = blockIdx.y, b = blockIdx.z;
  const int cs = gridDim.x, rank = blockIdx.x;         // the cluster spans grid x
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int gl = lane / 4, cl = lane % 4;
  const int G = L.H / L.H_kv;
  const int n = cache_len(L.c, L.H_kv, b, h, L.err);
  const int fresh = cache_new(L.n_new, L.n, b, L.err);
  const int rows = G * fresh;
  const int pos0 = L.c.next[b] - fresh;                // position of token 0
  const int near = static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(L.w) + fresh));
  uint8_t* ring = smem + warp * C::kWarpBytes;
  // The slots that the warp's pages keep, a ring of kList entries: page * 64 + row
  // and the scale exponents of K (low half) and V; with several tokens also the
  // position (kFar outside every window) and the group id.
  int2* list = reinterpret_cast<int2*>(ring + C::kRing);
  int2* about = list + (kMulti ? kList : 0);
  const int32_t* gids = L.gid + (static_cast<size_t>(b) * L.A + (L.A == 1 ? 0 : h)) * L.n;

  for (int r0 = 0; r0 < rows; r0 += C::kRows) {
    const int t_lo = r0 / G, tokens = (min(r0 + C::kRows, rows) - 1) / G - t_lo + 1;
    Scan<kBatch> scan;
    scan.first = warp * cs + rank;
    scan.step = kWarps * cs;
    scan.pages = (n + kPage - 1) / kPage;
    scan.n = n;
    scan.near_from = n - near;
    scan.k = 0;
    scan.fetch(L, b, h, lane);
    const int gid0 = gids[t_lo];
    if (kMulti) {
      if (threadIdx.x < tokens) s_gid[threadIdx.x] = gids[t_lo + threadIdx.x];
      __syncthreads();
    }

    // ---- query fragments, row factors, and the rows this thread's logits belong to
    uint32_t q[C::kParts][NT][C::kSteps][2];
    float factor[NT][2];
    int row_pos[NT][2], row_gid[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + gl;
      float x[C::kSteps][4];
      uint32_t top = 0;
      if (r < rows) {
        const T* src = static_cast<const T*>(L.Q) +
                       ((static_cast<size_t>(b) * L.H + h * G + r % G) * L.n + r / G) * D;
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) load4(src + (cl + 4 * (s / 4)) * 16 + (s % 4) * 4, x[s]);
      } else {
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) x[s][0] = x[s][1] = x[s][2] = x[s][3] = 0.f;
      }
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t u = __float_as_uint(x[s][e]) & 0x7fffffffu;
          if (u < 0x7f800000u) top = max(top, u);
        }
      top = max(top, __shfl_xor_sync(~0u, top, 1));
      top = max(top, __shfl_xor_sync(~0u, top, 2));
      const int eq = min(max(static_cast<int>(top >> 23) - 127 - 13, -110), 115);   // |q| 2^-eq < 2^14
      const float down = exp2_int(-eq);
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float lo = x[s][2 * e] * down, hi = x[s][2 * e + 1] * down;
          q[0][nt][s][e] = pack_half2(lo, hi);
          if (C::kParts == 2) {
            const float2 f = unpack_half2(q[0][nt][s][e]);
            q[C::kParts - 1][nt][s][e] = pack_half2(lo - f.x, hi - f.y);
          }
        }
      const float mine = exp2_int(eq) * L.scale_log2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        factor[nt][e] = __shfl_sync(~0u, mine, (2 * cl + e) * 4);
        const int rr = r0 + nt * 8 + 2 * cl + e;
        const int t = rr < rows ? rr / G : t_lo;
        row_pos[nt][e] = rr < rows ? pos0 + t : kFar;     // kFar: keeps nothing (see keeps)
        row_gid[nt][e] = kMulti ? s_gid[t - t_lo] : gid0;
      }
    }

    float o[NT][C::kSteps][4], ref[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ref[nt][e] = -INFINITY;
        sum[nt][e] = 0.f;
      }
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s) o[nt][s][0] = o[nt][s][1] = o[nt][s][2] = o[nt][s][3] = 0.f;
    }

    // Whether a query row at position i in group g keeps a listed slot.
    auto keeps = [&](int i, int g, const int2& slot) {
      return slot.x == kFar ? slot.y == g : cache_keep(i, slot.x, L.w, slot.y == g);
    };
    // Index of a listed slot in the pool's per-slot arrays.
    auto slot_at = [&](int row) {
      const uint32_t r = static_cast<uint32_t>(row);
      return (static_cast<size_t>(r / kPage) * L.H_kv + h) * kPage + r % kPage;
    };

    int entries = 0;
    // Appends the batch in registers to the list and fetches the next one.
    auto scan_batch = [&]() {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (scan.page[i] < 0) continue;
        const int j = scan.first + (scan.k + i) * scan.step;
        const int s = j * kPage + 2 * lane;
        const int id0 = static_cast<int16_t>(scan.ids[i] & 0xffffu), id1 = static_cast<int16_t>(scan.ids[i] >> 16);
        bool k0 = false, k1 = false;
        const bool window = (j + 1) * kPage > scan.near_from;
        for (int t = 0; t < (kMulti ? tokens : 1); ++t) {
          const int g = kMulti ? s_gid[t] : gid0;
          if (window) {
            k0 = k0 || cache_keep(pos0 + t_lo + t, scan.pos[i].x, L.w, id0 == g);
            k1 = k1 || cache_keep(pos0 + t_lo + t, scan.pos[i].y, L.w, id1 == g);
          } else {
            k0 = k0 || id0 == g;
            k1 = k1 || id1 == g;
          }
        }
        k0 = k0 && s < n;
        k1 = k1 && s + 1 < n;
        const uint32_t b0 = __ballot_sync(~0u, k0), b1 = __ballot_sync(~0u, k1);
        const uint32_t before = (1u << lane) - 1;
        const int at = entries + __popc(b0 & before) + __popc(b1 & before);
        const int row = scan.page[i] * kPage + 2 * lane;
        if (k0) {
          list[at & (kList - 1)] = make_int2(row, scan.exps[i]);
          if (kMulti) about[at & (kList - 1)] = make_int2(scan.pos[i].x, id0);
        }
        if (k1) {
          list[(at + k0) & (kList - 1)] = make_int2(row + 1, scan.exps[i]);
          if (kMulti) about[(at + k0) & (kList - 1)] = make_int2(scan.pos[i].y, id1);
        }
        entries += __popc(b0) + __popc(b1);
      }
      scan.k += kBatch;
      scan.fetch(L, b, h, lane);
      __syncwarp();
    };
    // Starts the copies of tile `tile` (rows past the list's end become zeros).
    auto issue = [&](int tile) {
      constexpr int kChunks = D / 16, kAtOnce = 32 / kChunks;
      if (tile * kKeys < entries) {
        uint8_t* stage = ring + (tile % kStages) * C::kStageBytes;
        const int c = lane % kChunks;
#pragma unroll
        for (int i = 0; i < kKeys / kAtOnce; ++i) {
          const int r = i * kAtOnce + lane / kChunks;
          const int idx = tile * kKeys + r;
          const bool there = idx < entries;
          const size_t off = slot_at(there ? list[idx & (kList - 1)].x : 0) * D + c * 16;
          // swizzles that spread a quarter warp's loads (below) over all banks
          const int kc = D == 128 ? c ^ ((r & 1) * 4) : c;
          const int vc = D == 128 ? c ^ (((r >> 1) & 3) * 2) : c ^ ((r >> 1) & 3);
          cp_async_16(stage + r * D + kc * 16, L.c.k + off, there ? 16 : 0);
          cp_async_16(stage + kKeys * D + r * D + vc * 16, L.c.v + off, there ? 16 : 0);
        }
      }
      cp_async_commit();
    };

    auto compute = [&](int tile) {
      const uint8_t* ks = ring + (tile % kStages) * C::kStageBytes;
      const uint8_t* vs = ks + kKeys * D;
      // S^T: two chains of products
      float acc[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) acc[nt][x][0] = acc[nt][x][1] = acc[nt][x][2] = acc[nt][x][3] = 0.f;
#pragma unroll
      for (int half = 0; half < D / 64; ++half) {
        const int c = cl + 4 * half, sw = D == 128 ? c ^ ((gl & 1) * 4) : c;   // gl + 8 has the same parity
        const uint4 lo = *reinterpret_cast<const uint4*>(ks + gl * D + sw * 16);
        const uint4 hi = *reinterpret_cast<const uint4*>(ks + (gl + 8) * D + sw * 16);
        const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a0 = e4m3x2_to_f16x2(static_cast<uint16_t>(lw[w]));
          const uint32_t a2 = e4m3x2_to_f16x2(static_cast<uint16_t>(lw[w] >> 16));
          const uint32_t a1 = e4m3x2_to_f16x2(static_cast<uint16_t>(hw[w]));
          const uint32_t a3 = e4m3x2_to_f16x2(static_cast<uint16_t>(hw[w] >> 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = 0; p < C::kParts; ++p)
              mma16816(acc[nt][w & 1], a0, a1, a2, a3, q[p][nt][half * 4 + w][0], q[p][nt][half * 4 + w][1]);
        }
      }
      // logits, masks and the reference
      const int i0 = tile * kKeys + gl;
      const int2 e0 = list[i0 & (kList - 1)], e1 = list[(i0 + 8) & (kList - 1)];
      const int2 m0 = about[i0 & (kList - 1)], m1 = about[(i0 + 8) & (kList - 1)];
      const bool in0 = i0 < entries, in1 = i0 + 8 < entries;
      const float kf0 = exp2_int(static_cast<int16_t>(e0.y & 0xffff)), kf1 = exp2_int(static_cast<int16_t>(e1.y & 0xffff));
      const int ve0 = e0.y >> 16, ve1 = e1.y >> 16;
      bool kept[NT][4];
      float t[NT][4];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int e = x & 1;
          bool on = (x < 2 ? in0 : in1) && row_pos[nt][e] != kFar;
          if (kMulti) on = on && keeps(row_pos[nt][e], row_gid[nt][e], x < 2 ? m0 : m1);
          kept[nt][x] = on;
          const float s = ((acc[nt][0][x] + acc[nt][1][x]) * factor[nt][e]) * (x < 2 ? kf0 : kf1);
          acc[nt][0][x] = s;
          t[nt][x] = s + static_cast<float>(x < 2 ? ve0 : ve1);
          grow = grow || (on && t[nt][x] > ref[nt][e] + 15.f);
        }
        if (L.logits) {
          float2* d0 = reinterpret_cast<float2*>(L.logits + slot_at(e0.x) * C::kRows + nt * 8 + 2 * cl);
          float2* d1 = reinterpret_cast<float2*>(L.logits + slot_at(e1.x) * C::kRows + nt * 8 + 2 * cl);
          if (in0) *d0 = make_float2(kept[nt][0] ? acc[nt][0][0] : -INFINITY, kept[nt][1] ? acc[nt][0][1] : -INFINITY);
          if (in1) *d1 = make_float2(kept[nt][2] ? acc[nt][0][2] : -INFINITY, kept[nt][3] ? acc[nt][0][3] : -INFINITY);
        }
      }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(kept[nt][e] ? t[nt][e] : -INFINITY, kept[nt][2 + e] ? t[nt][2 + e] : -INFINITY);
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
            if (top > ref[nt][e] + 15.f) {          // by the row's own weights: rows do not touch each other
              const float fresh_ref = top - 7.f, f = exp2f(ref[nt][e] - fresh_ref);
              ref[nt][e] = fresh_ref;
              sum[nt][e] *= f;
#pragma unroll
              for (int s = 0; s < C::kSteps; ++s) {
                o[nt][s][e] *= f;
                o[nt][s][2 + e] *= f;
              }
            }
          }
      }
      uint32_t pb[C::kParts][NT][2];
      const float vf0 = exp2_int(-ve0), vf1 = exp2_int(-ve1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          p[x] = kept[nt][x] ? exp2f(t[nt][x] - ref[nt][x & 1]) : 0.f;
          if (kept[nt][x]) sum[nt][x & 1] += p[x] * (x < 2 ? vf0 : vf1);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t hp = pack_half2(p[2 * x], p[2 * x + 1]);
          pb[0][nt][x] = transpose8x8(hp);
          if (C::kParts == 2) {
            const float2 f = unpack_half2(hp);
            pb[C::kParts - 1][nt][x] = transpose8x8(pack_half2(p[2 * x] - f.x, p[2 * x + 1] - f.y));
          }
        }
      }
      // O^T: thread (gl, cl) holds columns gl * D / 8 ... of keys 2 cl, 2 cl + 1, 2 cl + 8, 2 cl + 9
      uint32_t v[4][D / 32];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = 2 * cl + (x & 1) + (x >> 1) * 8;
        if (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(vs + r * D + (gl ^ (((r >> 1) & 3) * 2)) * 16);
          v[x][0] = u.x; v[x][1] = u.y; v[x][D / 32 - 2] = u.z; v[x][D / 32 - 1] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(vs + r * D + ((gl >> 1) ^ ((r >> 1) & 3)) * 16 + (gl & 1) * 8);
          v[x][0] = u.x; v[x][1] = u.y;
        }
      }
      uint32_t nan_keys = 0;                 // kMulti: bit x: this thread's piece of key x holds a NaN
      if (kMulti) {
        // A row that does not keep a key has weight 0 for it, and 0 * NaN would
        // reach that row: NaN codes leave the product and are put in afterwards.
        uint32_t any = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int w = 0; w < D / 32; ++w) any |= __vcmpeq4(v[x][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        if (__any_sync(~0u, any != 0)) {
          nan_keys = 1;
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) v[x][w] &= ~__vcmpeq4(v[x][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t sel = z ? 0x7362u : 0x5140u;
          const uint32_t u0 = __byte_perm(v[0][w], v[1][w], sel), u1 = __byte_perm(v[2][w], v[3][w], sel);
          const uint32_t a0 = e4m3x2_to_f16x2(static_cast<uint16_t>(u0));
          const uint32_t a1 = e4m3x2_to_f16x2(static_cast<uint16_t>(u0 >> 16));
          const uint32_t a2 = e4m3x2_to_f16x2(static_cast<uint16_t>(u1));
          const uint32_t a3 = e4m3x2_to_f16x2(static_cast<uint16_t>(u1 >> 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = 0; p < C::kParts; ++p)
              mma16816(o[nt][2 * w + z], a0, a1, a2, a3, pb[p][nt][0], pb[p][nt][1]);
        }
      if (kMulti && nan_keys) {
        // o[nt][s][x]: column gl * D / 8 + 2 s + x / 2 of row 2 cl + x % 2
        for (int r = 0; r < kKeys; ++r) {
          const int idx = tile * kKeys + r;
          if (idx >= entries) break;
          const int2 k = about[idx & (kList - 1)];
#pragma unroll
          for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int col = gl * (D / 8) + 2 * s + x / 2;
              const int c = D == 128 ? (col >> 4) ^ (((r >> 1) & 3) * 2) : (col >> 4) ^ ((r >> 1) & 3);
              if ((vs[r * D + c * 16 + (col & 15)] & 127) != 127) continue;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const int i = row_pos[nt][x & 1], g = row_gid[nt][x & 1];
                if (i != kFar && keeps(i, g, k)) o[nt][s][x] = __int_as_float(0x7fffffff);
              }
            }
        }
      }
    };

    // ---- the warp's pages
    auto fill = [&](int tile) {              // list every slot of tile `tile` that there is
      while (entries < (tile + 1) * kKeys && !scan.done()) scan_batch();
    };
#pragma unroll
    for (int x = 0; x < kStages - 1; ++x) {
      fill(x);
      issue(x);
    }
    for (int tile = 0;; ++tile) {
      fill(tile + kStages - 1);
      if (tile * kKeys >= entries) break;
      issue(tile + kStages - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      compute(tile);
      __syncwarp();                          // the stage is free for the next copies
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- join the block's warps
    float* part = reinterpret_cast<float*>(ring);          // [rows][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = sum[nt][e];
        l += __shfl_xor_sync(~0u, l, 4);
        l += __shfl_xor_sync(~0u, l, 8);
        l += __shfl_xor_sync(~0u, l, 16);
        const int r = nt * 8 + 2 * cl + e;
        if (gl == 0) {
          s_m[warp][r] = ref[nt][e];
          s_l[warp][r] = l;
        }
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s)
          *reinterpret_cast<float2*>(part + r * D + gl * (D / 8) + 2 * s) = make_float2(o[nt][s][e], o[nt][s][2 + e]);
      }
    }
    __syncthreads();
    // A warp without kept slots has sum 0 and is left out (its reference is -inf);
    // a NaN sum is not 0 and carries on.
    float4 mine[NT * D / 128 > 0 ? NT * D / 128 : 1];
    constexpr int kItems = C::kRows * D / 4;               // float4 pieces of the row block
#pragma unroll
    for (int x = 0; x < (kItems + kThreads - 1) / kThreads; ++x) {
      const int i = threadIdx.x + x * kThreads;
      if (i >= kItems) break;
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float M = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (s_l[w][r] == 0.f) continue;
        const float f = exp2f(s_m[w][r] - M);
        const float4 u = *reinterpret_cast<const float4*>(smem + w * C::kWarpBytes + (r * D + c) * 4);
        l += s_l[w][r] * f;
        a.x += u.x * f; a.y += u.y * f; a.z += u.z * f; a.w += u.w * f;
      }
      mine[x] = a;
      if (c == 0) {
        s_M[r] = M;
        s_L[r] = l;
      }
    }
    __syncthreads();
    float* whole = reinterpret_cast<float*>(smem);         // the block's partial, in warp 0's ring
#pragma unroll
    for (int x = 0; x < (kItems + kThreads - 1) / kThreads; ++x) {
      const int i = threadIdx.x + x * kThreads;
      if (i < kItems) *reinterpret_cast<float4*>(whole + 4 * i) = mine[x];
    }

    // ---- join the cluster's blocks; each writes its share of the rows
    cg::cluster_group cluster = cg::this_cluster();
    if (cs > 1) cluster.sync(); else __syncthreads();
    if (threadIdx.x < C::kRows) {
      const int r = threadIdx.x;
      float M = -INFINITY, l = 0.f;
      for (int x = 0; x < cs; ++x) M = fmaxf(M, cs > 1 ? *cluster.map_shared_rank(&s_M[r], x) : s_M[r]);
      for (int x = 0; x < cs; ++x) {
        const float m = cs > 1 ? *cluster.map_shared_rank(&s_M[r], x) : s_M[r];
        const float y = cs > 1 ? *cluster.map_shared_rank(&s_L[r], x) : s_L[r];
        if (y != 0.f) l += y * exp2f(m - M);
      }
      s_lse[r] = l != 0.f ? M + log2f(l) : -INFINITY;
      if (rank == 0 && L.lse && r0 + r < rows) {
        const int g = (r0 + r) % G, t = (r0 + r) / G;
        L.lse[(static_cast<size_t>(b) * L.H + h * G + g) * L.n + t] = s_lse[r] * 0.6931471805599453f;
      }
    }
    __syncthreads();
    const int share = (kItems + cs - 1) / cs;
    for (int i = rank * share + threadIdx.x; i < min(kItems, (rank + 1) * share); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      if (r0 + r >= rows) break;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = 0; x < cs; ++x) {
        const float m = cs > 1 ? *cluster.map_shared_rank(&s_M[r], x) : s_M[r];
        const float y = cs > 1 ? *cluster.map_shared_rank(&s_L[r], x) : s_L[r];
        if (y == 0.f) continue;
        const float4 u = *reinterpret_cast<const float4*>((cs > 1 ? cluster.map_shared_rank(whole, x) : whole) + 4 * i);
        const float f = exp2f(m - s_lse[r]);
        a.x += u.x * f; a.y += u.y * f; a.z += u.z * f; a.w += u.w * f;
      }
      const int g = (r0 + r) % G, t = (r0 + r) / G;
      store4(static_cast<T*>(L.O) + ((static_cast<size_t>(b) * L.H + h * G + g) * L.n + t) * D + c, a);
    }

    // ---- weights of the kept slots
    if (L.logits) {
      auto add = [&](int idx) {
        const size_t at = slot_at(list[idx & (kList - 1)].x);
        const float4* s = reinterpret_cast<const float4*>(L.logits + at * C::kRows);
        float w = 0.f;
#pragma unroll
        for (int x = 0; x < C::kRows / 4; ++x) {
          const float4 u = s[x];
          const float f[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (f[e] != -INFINITY) w += exp2f(f[e] - s_lse[4 * x + e]);
        }
        L.c.mass[at] += w;
      };
      if (entries <= kList) {                // the whole list is still there
        for (int i = lane; i < entries; i += 32) add(i);
      } else {
        int done = 0;
        entries = 0;
        scan.k = 0;
        scan.fetch(L, b, h, lane);
        while (done < entries || !scan.done()) {
          if (!scan.done()) scan_batch();
          for (int i = done + lane; i < entries; i += 32) add(i);
          done = entries;
          __syncwarp();
        }
      }
    }
    if (cs > 1) cluster.sync(); else __syncthreads();      // shared memory is read by others until here
  }
}

template <typename T, int D, int NT, bool kMulti>
cudaError_t launch(const CacheAttnLaunch& L, int cs, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cs, L.H_kv, L.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<T, D, NT, kMulti>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_kernel<T, D, NT, kMulti>, L);
}

template <typename T, int D>
cudaError_t launch_rows(const CacheAttnLaunch& L, int cs, cudaStream_t st) {
  const bool wide = cache_logit_rows(L.H / L.H_kv, L.n) == 16;
  if (L.n == 1) return wide ? launch<T, D, 2, false>(L, cs, st) : launch<T, D, 1, false>(L, cs, st);
  return wide ? launch<T, D, 2, true>(L, cs, st) : launch<T, D, 1, true>(L, cs, st);
}

template <typename T, int D, int NT, bool kMulti>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<T, D, NT, kMulti>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<T, D, NT, kMulti>::kSmem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(cache_attn_kernel<T, D, NT, kMulti>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

template <typename T, int D>
cudaError_t prepare_all() {
  if (cudaError_t e = prepare<T, D, 1, false>()) return e;
  if (cudaError_t e = prepare<T, D, 1, true>()) return e;
  if (cudaError_t e = prepare<T, D, 2, false>()) return e;
  return prepare<T, D, 2, true>();
}

}  // namespace

cudaError_t setup_cache_kernels() {
  if (cudaError_t e = prepare_all<__nv_bfloat16, 64>()) return e;
  if (cudaError_t e = prepare_all<__nv_bfloat16, 128>()) return e;
  if (cudaError_t e = prepare_all<float, 64>()) return e;
  return prepare_all<float, 128>();
}

cudaError_t launch_cache_attn(const CacheAttnLaunch& L, int dtype, cudaStream_t st) {
  // Blocks per (sequence, head): enough that every SM has two, as long as each
  // warp gets a page.
  int cs = 1;
  while (cs < 16 && cs * L.B * L.H_kv < 2 * L.num_sms && cs * kWarps < L.c.max_pages) cs *= 2;
  if (dtype == FOCUS_BF16) return L.d == 128 ? launch_rows<__nv_bfloat16, 128>(L, cs, st) : launch_rows<__nv_bfloat16, 64>(L, cs, st);
  return L.d == 128 ? launch_rows<float, 128>(L, cs, st) : launch_rows<float, 64>(L, cs, st);
}

}  // namespace focus
