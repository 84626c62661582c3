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
// and gathers their rows in tiles of 16 keys with cp.async, a tile ahead of the
// products.  Only kept rows are read.
//
// Products run on mma.sync with the keys on the 16 side and the query rows
// (tokens x query heads of the head) on the 8 side:
//   S^T = K Q^T:    thread (g, c) = (lane / 4, lane % 4) holds row g of the key
//                   fragment.  The sum over d may run in any order, so the thread
//                   takes 16 consecutive bytes of its row and Q is laid out to
//                   match: no transposition, one 16-byte load per 16 codes.
//   O^T += V^T P^T: two keys' bytes of one column are zipped with one byte
//                   permute into the pairs that the fragment wants; P^T comes
//                   from S^T by an 8x8 register transpose.
// Codes become f16 exactly and the products run in f16 with fp32 sums (an e4m3
// m16n8k32 of mma.sync is two f16 products here as well, by the counters of a probe).
// Queries are scaled by a power of two per row to below 2^14 and held in one f16
// (bf16 tensors: 8 bits fit 11) or two (fp32 tensors, 22 bits); weights are held in
// two, since one alone would be off by up to 2^-11, an eighth of bf16's half step.
//
// Softmax: with v = code * 2^e per page, the running maximum is taken over
// t_j = s_j + e_j (log2), so the weights 2^(t_j - ref) multiply raw codes and
// stay in range for pages of any scale; the row sum adds 2^(t_j - ref) 2^-e_j in
// fp32, or 2^(s_j - ref) where the scales lie far apart (kScaleSpan).  ref lies 7
// below the maximum when it is set and is moved only when a weight would pass 2^15,
// so f16's subnormals begin 2^-21 below the largest one.
//
// The warps' partials are joined in shared memory; each block then sends every
// other block of the cluster the part of the rows that that one writes.
// With accumulate a second pass over the listed slots, when the rows' sums are
// known, forms the logits again from K (d bytes a kept slot; keeping them would
// cost 8 bytes a slot and query row) and adds each slot's weights: one addition
// a slot, in a fixed order.
//
// Measured: one step of 32 / 8 heads over 32K slots 11.0 us; 16 sequences of up to 32K
// 57 us with the weights accumulated (86 MB: 1.5 TB/s; 54 with weights of one f16); a step of 8 sequences of up to
// 1K slots, 12 heads, d = 64, 8.4 us.
// The two small ones are a chain of latencies: launch, counts and table, group ids,
// rows, products, two joins (18,400 clocks at 32K: first tile there at 10,200,
// products done at 13,100, cluster joined at 16,200).  The batch runs at 47% of the
// issue rate with 13% of the DRAM rate: two blocks an SM do not hide the latencies
// of a block, the sequences are uneven, and the second pass takes a third of a block's
// time (47,700 clocks to the join, 22,600 after it).
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
constexpr int kMaxCluster = kMaxClusterBlocks;
constexpr int kAhead = 16;           // pages whose group ids a warp holds in shared memory
constexpr int kList = 256;           // entries of a warp's list of kept slots
// Sums are held times 2^kLift.  s_max - ref lies within [7 - 120, 15 + 64], so a row's
// largest term within 2^-96 and 2^96: 2^30 slots of it do not overflow, and a term is
// lost only below 2^-30 of it.
constexpr int kLift = 17;
static_assert(kList >= kPage + (kStages + 1) * kKeys && (kList & (kList - 1)) == 0, "list too short");

template <typename T, int D, int NT>
struct Cfg {
  static constexpr int kParts = std::is_same<T, float>::value ? 2 : 1;   // f16 parts of q; of P there are two
  static constexpr int kRows = 8 * NT;
  static constexpr int kSteps = D / 16;                                  // f16 MMA steps over d
  static constexpr int kStageBytes = 2 * kKeys * D;                      // K rows, then V rows
  // A warp's region: the tile ring, later its partial result (rows 16 bytes apart
  // modulo 64, so that a fragment's stores fall on different banks), the list and
  // the group ids.
  static constexpr int kPitch = D * 4 + 16;
  static constexpr int kRing = kStages * kStageBytes > kRows * kPitch ? kStages * kStageBytes : kRows * kPitch;
  static constexpr int kWarpBytes = kRing + kList * 8 + kAhead * kPage * 2;
  static constexpr int kItems = kRows * D / 4;                           // float4 pieces of a row block's result
  static constexpr int kInbox = (kItems + kMaxCluster) * 16;             // pieces of every block of the cluster
  static constexpr int kSmem = kWarps * kWarpBytes + 2 * kInbox;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
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
__device__ __forceinline__ void store2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x, y);
}

template <typename T, int D, int NT, bool kMulti>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) cache_attn_kernel(CacheAttnLaunch L) {
  using C = Cfg<T, D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];   // the warps' references and sums per row
  __shared__ float2 s_all[2][kMaxCluster][C::kRows];   // ... and the cluster's blocks'
  __shared__ float s_factor[kMaxCluster][C::kRows];    // weight of a block's partial in the row
  __shared__ float s_lse[C::kRows];                    // log2 sum-exp of the whole row
  __shared__ int s_gid[C::kRows];                      // group id of each token of the row block
  cg::cluster_group cluster = cg::this_cluster();
  // Every block of the cluster has to run before another writes into it: waited
  // for at the first join.
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int h = blockIdx.y, b = blockIdx.z;
  const int cs = gridDim.x, rank = blockIdx.x;         // the cluster spans grid x
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int gl = lane / 4, cl = lane % 4;
  const int G = L.H / L.H_kv;
  uint8_t* ring = smem + warp * C::kWarpBytes;
  // Kept slots: x = first 16-byte piece of the slot's row in the pool, y = scale
  // exponents of K and V (bytes 0 and 1) and a bit for each token that keeps it.
  int2* list = reinterpret_cast<int2*>(ring + C::kRing);
  uint32_t* ids = reinterpret_cast<uint32_t*>(ring + C::kRing + kList * 8);
  uint8_t* inbox = smem + kWarps * C::kWarpBytes;
  const int32_t* gids = L.gid + (static_cast<size_t>(b) * L.A + (L.A == 1 ? 0 : h)) * L.n;
  const int first = warp * cs + rank, step = kWarps * cs;          // the warp's pages
  // Units of the scan: pages, and from page `split` on (where every slot of a window
  // lies, if the windows' pages are fewer than the warps) quarters of pages, so that
  // no warp gets four tiles while most get one.
  int n = 0, fresh = 0, pos0 = 0, units = 0, near_from = 0, split = INT_MAX;
  auto page_of = [&](int u) { return u < split ? u : split + (u - split) / 4; };
  auto table = [&](int from) {                         // table entry of the lane's unit among kAhead, unchecked
    const int j = page_of(from + lane * step);
    return lane < kAhead && j < L.c.max_pages ? L.c.table[static_cast<size_t>(b) * L.c.max_pages + j] : -1;
  };
  int rows = G;                                        // set in the first round, which always runs

  int buf = 0;
  for (int r0 = 0; r0 < rows; r0 += C::kRows, buf ^= 1) {
    // ---- loads that depend on nothing go first: table (as if without quarters), group
    // ids, query rows, counts
    int entry = table(first);
    const int t_lo = r0 / G;
    const int gid0 = gids[t_lo];
    int gid_mine = 0;
    if (kMulti && threadIdx.x < C::kRows && t_lo + threadIdx.x < L.n) gid_mine = gids[t_lo + threadIdx.x];
    float x[NT][C::kSteps][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + gl;
      if (r < G * L.n) {
        const T* src = static_cast<const T*>(L.Q) +
                       ((static_cast<size_t>(b) * L.H + h * G + r % G) * L.n + r / G) * D;
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) load4(src + (cl + 4 * (s / 4)) * 16 + (s % 4) * 4, x[nt][s]);
      } else {
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) x[nt][s][0] = x[nt][s][1] = x[nt][s][2] = x[nt][s][3] = 0.f;
      }
    }
    if (r0 == 0) {
      n = cache_len(L.c, L.H_kv, b, h, L.err);
      fresh = cache_new(L.n_new, L.n, b, L.err);
      pos0 = L.c.next[b] - fresh;                      // position of token 0
      rows = G * fresh;
      const int pages = (n + kPage - 1) / kPage;
      near_from = n - static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(L.w) + fresh));
      split = near_from / kPage;
      if (pages - split > step) split = pages;
      units = split + 4 * (pages - split);
      if (rows == 0) break;                            // the same in the whole cluster
      if (first + lane * step > split) entry = table(first);       // another page than the guess
    }
    const int tokens = (min(r0 + C::kRows, rows) - 1) / G - t_lo + 1;

    // ---- the scan: kAhead pages at a time, their group ids in shared memory
    int j = first, i = 0;                              // next unit to scan, and its place among the kAhead
    int lane_page = -1, lane_exps = 0;
    PageScales scales{1.f, 1.f};
    int2 pos{};                                        // positions of the lane's two slots of unit j, if it is near
    auto load_pos = [&]() {
      const int page = __shfl_sync(~0u, lane_page, i);
      if (page >= 0 && (page_of(j) + 1) * kPage > near_from)
        pos = *reinterpret_cast<const int2*>(L.c.pos + (static_cast<size_t>(page) * L.H_kv + h) * kPage + 2 * lane);
    };
    auto open_pages = [&]() {                          // units j, j + step, ...
      i = 0;
      lane_page = -1;
      if (lane < kAhead && j + lane * step < units) {
        lane_page = entry;
        if (entry < 0 || entry >= L.c.n_pages) {
          atomicOr(L.err, kErrBadCache);
          lane_page = -1;
        }
      }
#pragma unroll
      for (int x = 0; x < kAhead * kPage * 2 / 16 / 32; ++x) {
        const int page = __shfl_sync(~0u, lane_page, x * 4 + lane / 8);
        if (page >= 0)
          cp_async_16(ids + x * 128 + lane * 4,
                      L.c.gid + (static_cast<size_t>(page) * L.H_kv + h) * kPage + lane % 8 * 8, 16);
      }
      if (lane_page >= 0) scales.load(L.c, static_cast<size_t>(lane_page) * L.H_kv + h);
      entry = table(j + kAhead * step);
      load_pos();
    };
    open_pages();
    if (kMulti) {
      if (threadIdx.x < C::kRows) s_gid[threadIdx.x] = gid_mine;
      __syncthreads();
    }

    // ---- query fragments, row factors, and the rows this thread's logits belong to
    uint32_t q[C::kParts][NT][C::kSteps][2];
    float factor[NT][2];
    int row_bit[NT][2];                                // bit of the row's token in a list entry, 0: no such row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t top = 0;
      bool finite = true;
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t u = __float_as_uint(x[nt][s][e]) & 0x7fffffffu;
          if (u < 0x7f800000u) top = max(top, u);
          else finite = false;
        }
      // rows with an infinite or NaN element become NaN through their factor
      finite = (__ballot_sync(~0u, finite) >> (lane & ~3) & 15) == 15;
      top = max(top, __shfl_xor_sync(~0u, top, 1));
      top = max(top, __shfl_xor_sync(~0u, top, 2));
      const int eq = min(max(static_cast<int>(top >> 23) - 127 - 13, kMinQueryExp), 115);   // |q| 2^-eq < 2^14
      const float down = exp2_int(-eq);
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float lo = x[nt][s][2 * e] * down, hi = x[nt][s][2 * e + 1] * down;
          q[0][nt][s][e] = pack_half2(lo, hi);
          if constexpr (C::kParts == 2) {
            const float2 f = unpack_half2(q[0][nt][s][e]);
            q[1][nt][s][e] = pack_half2(lo - f.x, hi - f.y);
          }
        }
      const float mine = finite ? exp2_int(eq) * L.scale_log2 : __int_as_float(0x7fffffff);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        factor[nt][e] = __shfl_sync(~0u, mine, (2 * cl + e) * 4);
        const int rr = r0 + nt * 8 + 2 * cl + e;
        row_bit[nt][e] = rr < rows ? static_cast<int>(0x10000u << (kMulti ? rr / G - t_lo : 0)) : 0;
      }
    }

    float o[NT][C::kSteps][4], ref[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ref[nt][e] = kNoRef;
        sum[nt][e] = 0.f;
      }
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s) o[nt][s][0] = o[nt][s][1] = o[nt][s][2] = o[nt][s][3] = 0.f;
    }

    int entries = 0;
    int e_top = kMinExp, e_bot = kMaxExp;              // value exponents of the pages opened so far
    // Lists the kept slots of unit j.
    auto scan_page = [&]() {
      if (i == 0) {                                    // new group ids have to have landed
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();
        lane_exps = scales.bytes();
        const int ve = static_cast<int8_t>(lane_exps >> 8);
        e_top = max(e_top, __reduce_max_sync(~0u, lane_page >= 0 ? ve : kMinExp));
        e_bot = min(e_bot, __reduce_min_sync(~0u, lane_page >= 0 ? ve : kMaxExp));
      }
      const int page = __shfl_sync(~0u, lane_page, i), exps = __shfl_sync(~0u, lane_exps, i);
      if (page >= 0) {
        const uint32_t two = ids[i * 32 + lane];
        const int from = page_of(j) * kPage;
        const bool near = from + kPage > near_from;
        int m0 = 0, m1 = 0;
        for (int t = 0; t < (kMulti ? tokens : 1); ++t) {
          const int g = kMulti ? s_gid[t] : gid0, p = pos0 + t_lo + t;
          bool k0 = static_cast<int16_t>(two & 0xffffu) == g, k1 = static_cast<int16_t>(two >> 16) == g;
          if (near) {
            k0 = cache_keep(p, pos.x, L.w, k0);
            k1 = cache_keep(p, pos.y, L.w, k1);
          }
          m0 |= k0 << t;
          m1 |= k1 << t;
        }
        if (from + kPage > n) {
          const int left = n - from - 2 * lane;
          if (left < 1) m0 = 0;
          if (left < 2) m1 = 0;
        }
        if (j >= split && lane / 8 != ((j - split) & 3)) m0 = m1 = 0;      // another quarter's
        const uint32_t b0 = __ballot_sync(~0u, m0 != 0), b1 = __ballot_sync(~0u, m1 != 0);
        if (b0 | b1) {
          const uint32_t before = (1u << lane) - 1;
          const int at = entries + __popc(b0 & before) + __popc(b1 & before);
          const uint32_t row = ((static_cast<uint32_t>(page) * L.H_kv + h) * kPage + 2 * lane) * (D / 16);
          if (m0) list[at & (kList - 1)] = make_int2(row, exps | m0 << 16);
          if (m1) list[(at + (m0 != 0)) & (kList - 1)] = make_int2(row + D / 16, exps | m1 << 16);
          entries += __popc(b0) + __popc(b1);
        }
      }
      j += step;
      ++i;
      __syncwarp();
      if (i == kAhead) open_pages(); else load_pos();
    };
    // Starts the copies of tile `tile` (rows past the list's end become zeros).  Pieces
    // are swizzled to spread a quarter warp's loads in compute() over all banks.
    constexpr int kChunks = D / 16, kAtOnce = 32 / kChunks;
    static_assert(kList % kKeys == 0, "a tile's entries are consecutive");
    const int lr = lane / kChunks, lc = lane % kChunks;
    const uint32_t to_k = lr * D + (D == 128 ? lc ^ (lr & 1) * 4 : lc) * 16;
    const uint32_t to_v = kKeys * D + lr * D + (D == 128 ? lc ^ (lr >> 1) * 2 : lc ^ (lr >> 1)) * 16;
    auto issue = [&](int tile, bool values) {
      const int left = entries - tile * kKeys;
      if (left > 0) {
        uint8_t* stage = ring + (tile % kStages) * C::kStageBytes;
        const int2* from = list + (tile * kKeys & (kList - 1)) + lr;
#pragma unroll
        for (int y = 0; y < kKeys / kAtOnce; ++y) {
          const bool there = left >= kKeys || lr + y * kAtOnce < left;
          const size_t off = static_cast<size_t>(static_cast<uint32_t>(there ? from[y * kAtOnce].x : 0) + lc) * 16;
          cp_async_16(stage + to_k + y * kAtOnce * D, L.c.k + off, there ? 16 : 0);
          // rows move on by kAtOnce: the value swizzle flips its upper bit with every odd y (d = 128)
          if (values)
            cp_async_16(stage + (to_v ^ (D == 128 ? (y & 1) * 64 : 0)) + y * kAtOnce * D, L.c.v + off, there ? 16 : 0);
        }
      }
      cp_async_commit();
    };

    // Products of tile `tile`; `last`: the pass that only adds up the slots' weights.
    auto compute = [&](int tile, bool last) {
      const uint8_t* ks = ring + (tile % kStages) * C::kStageBytes;
      const uint8_t* vs = ks + kKeys * D;
      // S^T: two chains of products
      float acc[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) acc[nt][y][0] = acc[nt][y][1] = acc[nt][y][2] = acc[nt][y][3] = 0.f;
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
              mma_f16(acc[nt][w & 1], a0, a1, a2, a3, q[p][nt][half * 4 + w][0], q[p][nt][half * 4 + w][1]);
        }
      }
      // logits; slots that a row does not keep: -inf
      const int2* about = list + (tile * kKeys & (kList - 1)) + gl;
      const int2 e0 = about[0], e1 = about[8];
      const int left = entries - tile * kKeys - gl;
      const int mask0 = left > 0 ? e0.y : 0, mask1 = left > 8 ? e1.y : 0;      // past the end: no row, scales 1
      const float kf0 = exp2_int(static_cast<int8_t>(mask0)), kf1 = exp2_int(static_cast<int8_t>(mask1));
      float t[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          t[nt][y] = ((acc[nt][0][y] + acc[nt][1][y]) * factor[nt][y & 1]) * (y < 2 ? kf0 : kf1);
          if (((y < 2 ? mask0 : mask1) & row_bit[nt][y & 1]) == 0) t[nt][y] = -INFINITY;
        }
      if (last) {
        float w0 = 0.f, w1 = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float lse = s_lse[nt * 8 + 2 * cl + e];      // a large number for rows without kept slots
            // rows that do not keep the slot add nothing, also where their sum is NaN
            w0 += mask0 & row_bit[nt][e] ? exp2_fast(t[nt][e] - lse) : 0.f;
            w1 += mask1 & row_bit[nt][e] ? exp2_fast(t[nt][2 + e] - lse) : 0.f;
          }
        w0 += __shfl_xor_sync(~0u, w0, 1);
        w1 += __shfl_xor_sync(~0u, w1, 1);
        w0 += __shfl_xor_sync(~0u, w0, 2);
        w1 += __shfl_xor_sync(~0u, w1, 2);
        // the only addition to this slot for these rows: its order cannot matter
        if (cl == 0 && left > 0) atomicAdd(L.c.mass + static_cast<uint32_t>(e0.x) / (D / 16), w0);
        if (cl == 1 && left > 8) atomicAdd(L.c.mass + static_cast<uint32_t>(e1.x) / (D / 16), w1);
        return;
      }
      // the weights' reference
      const int ve0 = static_cast<int8_t>(mask0 >> 8), ve1 = static_cast<int8_t>(mask1 >> 8);
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          t[nt][y] += static_cast<float>(y < 2 ? ve0 : ve1);
          grow = grow || t[nt][y] > ref[nt][y & 1] + 15.f;
        }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(t[nt][e], t[nt][2 + e]);
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
            if (top > ref[nt][e] + 15.f) {          // by the row's own weights: rows do not touch each other
              // in two steps: the factor may lie below the normals where the sum does not
              const float moved = top - 7.f, fh = exp2_fast(0.5f * (ref[nt][e] - moved)), f = fh * fh;
              ref[nt][e] = moved;
              sum[nt][e] = sum[nt][e] * fh * fh;
#pragma unroll
              for (int s = 0; s < C::kSteps; ++s) {
                o[nt][s][e] *= f;
                o[nt][s][2 + e] *= f;
              }
            }
          }
      }
      uint32_t pb[2][NT][2];                        // [part][..][keys 0-7 or 8-15]
      float vf0 = exp2_int(kLift - ve0), vf1 = exp2_int(kLift - ve1);
      if (e_top - e_bot > kScaleSpan) {              // the same in the whole warp
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            sum[nt][y & 1] += exp2_fast(t[nt][y] - ref[nt][y & 1] + static_cast<float>(kLift - (y < 2 ? ve0 : ve1)));
        vf0 = vf1 = 0.f;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          p[y] = exp2_fast(t[nt][y] - ref[nt][y & 1]);
          sum[nt][y & 1] = fmaf(p[y], y < 2 ? vf0 : vf1, sum[nt][y & 1]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t hp = pack_half2(p[2 * y], p[2 * y + 1]);
          pb[0][nt][y] = transpose8x8(hp);
          const float2 f = unpack_half2(hp);
          pb[1][nt][y] = transpose8x8(pack_half2(p[2 * y] - f.x, p[2 * y + 1] - f.y));
        }
      }
      // O^T: thread (gl, cl) holds columns gl * D / 8 ... of keys 2 cl, 2 cl + 1, 2 cl + 8, 2 cl + 9
      uint32_t v[4][D / 32];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int r = 2 * cl + (y & 1) + (y >> 1) * 8;
        if (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(vs + r * D + (gl ^ (((r >> 1) & 3) * 2)) * 16);
          v[y][0] = u.x; v[y][1] = u.y; v[y][D / 32 - 2] = u.z; v[y][D / 32 - 1] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(vs + r * D + ((gl >> 1) ^ ((r >> 1) & 3)) * 16 + (gl & 1) * 8);
          v[y][0] = u.x; v[y][1] = u.y;
        }
      }
      bool some_nan = false;                 // the same in the whole warp
      if (kMulti) {
        // A row that does not keep a key has weight 0 for it, and 0 * NaN would
        // reach that row: NaN codes leave the product and are put in afterwards.
        uint32_t any = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int w = 0; w < D / 32; ++w) any |= __vcmpeq4(v[y][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        some_nan = __any_sync(~0u, any != 0);
        if (some_nan) {
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) v[y][w] &= ~__vcmpeq4(v[y][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
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
            for (int p = 0; p < 2; ++p)
              mma_f16(o[nt][2 * w + z], a0, a1, a2, a3, pb[p][nt][0], pb[p][nt][1]);
        }
      if (kMulti && some_nan) {
        // o[nt][s][y]: column gl * D / 8 + 2 s + y / 2 of row 2 cl + y % 2
        for (int r = 0; r < kKeys && tile * kKeys + r < entries; ++r) {
          const int mask = list[(tile * kKeys + r) & (kList - 1)].y;
#pragma unroll
          for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int col = gl * (D / 8) + 2 * s + y / 2;
              const int c = D == 128 ? (col >> 4) ^ (((r >> 1) & 3) * 2) : (col >> 4) ^ ((r >> 1) & 3);
              if ((vs[r * D + c * 16 + (col & 15)] & 127) != 127) continue;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                if (mask & row_bit[nt][y & 1]) o[nt][s][y] = __int_as_float(0x7fffffff);
            }
        }
      }
    };

    for (int pass = 0; pass < (L.accumulate ? 2 : 1); ++pass) {
      if (pass == 1) {
        if (entries > kList) {               // the list's start is gone: scan again
          entries = 0;
          j = first;
          entry = table(first);
          open_pages();
        }
      }
      // ---- the warp's pages: copies run kStages - 1 tiles ahead of the products
      for (int tile = 1 - kStages;; ++tile) {
        while (entries < (tile + kStages) * kKeys && j < units) scan_page();
        if (tile >= 0 && tile * kKeys >= entries) break;
        issue(tile + kStages - 1, pass == 0);
        if (tile < 0) continue;
        cp_async_wait<kStages - 1>();
        __syncwarp();
        compute(tile, pass == 1);
        __syncwarp();                        // the stage is free for the next copies
      }
      cp_async_wait<0>();
      __syncwarp();
      if (pass == 1) break;

      // ---- join the block's warps.  A piece j of a row holds columns 2 s, 2 s + 1 of the
      // D / 8 columns of two neighbouring gl: s = j / 4, gl = 2 (j % 4) and the next.
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
            *reinterpret_cast<float2*>(ring + r * C::kPitch + s * 64 + gl * 8) = make_float2(o[nt][s][e], o[nt][s][2 + e]);
        }
      }
      if (r0 == 0) asm volatile("barrier.cluster.wait;" ::: "memory");
      __syncthreads();
      // Pieces of one share go to one block's inbox, which that block joins and writes:
      // stores into another block's memory are not waited for, loads from it would be.
      // A warp without kept slots has sum 0 and is left out;
      // a NaN sum is not 0 and carries on.
      const int share = (C::kItems + cs - 1) / cs;
  #pragma unroll
      for (int y = 0; y < (C::kItems + kThreads - 1) / kThreads; ++y) {
        const int i = threadIdx.x + y * kThreads;
        if (i >= C::kItems) break;
        const int r = i / (D / 4), j = i % (D / 4);
        float M = -INFINITY, l = 0.f;
  #pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  #pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 u = *reinterpret_cast<const float4*>(smem + w * C::kWarpBytes + r * C::kPitch + j * 16);
          if (s_l[w][r] == 0.f) continue;
          const float fh = exp2f(0.5f * (s_m[w][r] - M)), f = fh * fh;   // two steps for the sum, as above
          l += s_l[w][r] * fh * fh;
          a.x += u.x * f; a.y += u.y * f; a.z += u.z * f; a.w += u.w * f;
        }
        const int to = i / share;
        float4* box = reinterpret_cast<float4*>(inbox + buf * C::kInbox) + rank * share + (i - to * share);
        *cluster.map_shared_rank(box, to) = a;
        if (j < cs) *cluster.map_shared_rank(&s_all[buf][rank][r], j) = make_float2(M, l);
      }

      // ---- join the cluster's blocks
      cluster.sync();
      if (threadIdx.x < kMaxCluster * C::kRows) {           // 16 lanes a row, one a block
        const int from = threadIdx.x % kMaxCluster, r = threadIdx.x / kMaxCluster;
        const float2 v = from < cs ? s_all[buf][from][r] : make_float2(-INFINITY, 0.f);
        float M = v.x;
  #pragma unroll
        for (int y = 8; y > 0; y /= 2) M = fmaxf(M, __shfl_xor_sync(~0u, M, y));
        const float fh = v.y != 0.f ? exp2f(0.5f * (v.x - M)) : 0.f, f = fh * fh;
        float l = v.y != 0.f ? v.y * fh * fh : 0.f;
  #pragma unroll
        for (int y = 8; y > 0; y /= 2) l += __shfl_xor_sync(~0u, l, y);
        s_factor[from][r] = v.y != 0.f ? f / l * exp2_int(kLift) : 0.f;
        if (from == 0) {
          const float lse = l != 0.f ? M + (log2f(l) - kLift) : -INFINITY;
          s_lse[r] = l != 0.f ? lse : -kNoRef;
          if (rank == 0 && L.lse && r0 + r < rows)
            L.lse[(static_cast<size_t>(b) * L.H + h * G + (r0 + r) % G) * L.n + (r0 + r) / G] = lse * 0.6931471805599453f;
        }
      }
      __syncthreads();
      for (int i = rank * share + threadIdx.x; i < min(C::kItems, (rank + 1) * share); i += kThreads) {
        const int r = i / (D / 4), j = i % (D / 4);
        if (r0 + r >= rows) break;
        const float4* box = reinterpret_cast<const float4*>(inbox + buf * C::kInbox) + (i - rank * share);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  #pragma unroll 4
        for (int from = 0; from < cs; ++from) {
          const float4 u = box[from * share];
          const float f = s_factor[from][r];
          if (f == 0.f) continue;                           // nothing kept there
          a.x += u.x * f; a.y += u.y * f; a.z += u.z * f; a.w += u.w * f;
        }
        T* out = static_cast<T*>(L.O) + ((static_cast<size_t>(b) * L.H + h * G + (r0 + r) % G) * L.n + (r0 + r) / G) * D +
                 j % 4 * (D / 4) + j / 4 * 2;
        store2(out, a.x, a.y);
        store2(out + D / 8, a.z, a.w);
      }
    }
    __syncthreads();                         // shared memory is free for the next row block
  }
  if (rows == 0) asm volatile("barrier.cluster.wait;" ::: "memory");
}

template <typename T, int D, int NT, bool kMulti>
ClusterFits g_fits;

template <typename T, int D, int NT, bool kMulti>
cudaError_t launch(const CacheAttnLaunch& L, cudaStream_t st) {
  // Blocks per (sequence, head): one wave of the clusters that fit, as long as each warp
  // gets a page.  In several waves 2 a head, and in up to two waves 4, where a warp still
  // has 8 pages for each wave, or 4 if they are read twice (accumulate): sequences differ
  // in what they keep, and a block's latencies hide behind others'.  Up to n pages for each
  // of B sequences of 8 heads, 4 rows, us with 1, 2, 4 blocks, in brackets with the weights
  // accumulated; * is taken:
  //   B = 16, n = 128:  25, 20*, 25 (42, 27*, 29)     256: 46, 28*, 26 (81, 47, 32*)
  //           n = 512:  61, 36, 32* (110, 62, 40*)    1024: 111, 62, 49* (203, 110, 77*)
  //   B = 32, n = 64:   21*, 28, 40 (29*, 36, 48)     128: 31*, 36, 46 (52, 45*, 56)
  //           n = 256:  44, 45*, 53 (74, 58*, 66)     1024: 167, 149*, 125 (306, 204*, 182)
  //   B = 64, n = 128:  58*, 58, 82 (87*, 76, 100)    512: 134, 109*, 128 (221, 170*, 167)
  // The table's size is what the launch knows: sequences much shorter than that lose by
  // more blocks what the figures for small n show, so four stay within two waves.
  const ClusterFit* fit;
  if (cudaError_t e = g_fits<T, D, NT, kMulti>.get(L.device, reinterpret_cast<const void*>(cache_attn_kernel<T, D, NT, kMulti>),
                                                   kThreads, Cfg<T, D, NT>::kSmem, &fit))
    return e;
  const long long heads = static_cast<long long>(L.B) * L.H_kv;
  int cs = 1, i = 0;
  while (cs < kMaxCluster && cs * kWarps < L.c.max_pages) {
    const int runs = fit->n[i + 1];
    const long long worth = static_cast<long long>(2 * cs * kWarps) * (L.accumulate ? 4 : 8);   // pages, for one wave
    const bool pays = heads * worth <= static_cast<long long>(L.c.max_pages) * runs;
    if (heads > runs && (!pays || cs > 2 || (cs == 2 && heads > 2 * runs))) break;
    cs *= 2;
    ++i;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cs, L.H_kv, L.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<T, D, NT>::kSmem;
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
cudaError_t launch_rows(const CacheAttnLaunch& L, cudaStream_t st) {
  const bool wide = L.H / L.H_kv * L.n > 8;
  if (L.n == 1) return wide ? launch<T, D, 2, false>(L, st) : launch<T, D, 1, false>(L, st);
  return wide ? launch<T, D, 2, true>(L, st) : launch<T, D, 1, true>(L, st);
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnLaunch& L, int dtype, cudaStream_t st) {
  if (dtype == FOCUS_BF16) return L.d == 128 ? launch_rows<__nv_bfloat16, 128>(L, st) : launch_rows<__nv_bfloat16, 64>(L, st);
  return L.d == 128 ? launch_rows<float, 128>(L, st) : launch_rows<float, 64>(L, st);
}

}  // namespace focus
