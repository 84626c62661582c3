// Focus attention of new tokens over the paged 8-bit cache on the tcgen05 tensor
// cores: bf16 tensors, d = 128, more than 16 query rows a head (contract: focus.h;
// cache_attn.cu has the form for every other case).
//
// The codes go into the products as they are, kind::f8f6f4, gathered into tiles of
// 128 kept slots with cp.async (TMA's row gather took 80 clocks for four rows, 6 B a
// clock and SM; a third of that is needed):
//   S^T [128 keys, 2 R]   = K Q^T      K rows K-major; Q as q = 2^e (q1 + q2 / 16) in
//                           e4m3, both parts side by side in N: 4 + 4 bits hold
//                           bf16's 8, elements below 2^-15 of a row's largest are
//                           held to 2^-23 of it
//   O^T [128 dims, 4 R] += V^T P^T     V rows are an MN-major A; P as p1 + p2 / 16 +
//                           p3 / 256 + p4 / 4096 in e4m3, again side by side in N
//                           with sums of their own: 2^-16 of a weight, and 2^-22
//                           where that is more, which is 2^-26 of a row's largest
//                           weight or less (see below)
// R = 32 or 64 query rows (tokens x query heads of the head; 16 or fewer are faster on
// mma.sync).  With the keys
// on the 128 side of both products nothing is padded but R, and a thread owns a
// key: masks, scales and the weight's sum over rows need no exchange.
//
// Work split, softmax reference and join are cache_attn.cu's: a cluster of blocks
// per (sequence, head), pages round-robin over the blocks.  In a block three or five
// warps scan group ids (and the last slots' positions) into a list of kept slots, in
// rounds, up to four tiles ahead; four gather the tiles; one issues the products;
// eight or sixteen (two or four a TMEM lane quadrant, each for a part of the rows)
// form the weights.  The reference of a row is common to the block: it is set kBelow
// below the largest t and moves only when a weight would pass 2^kTop, so the
// accumulator in TMEM is rescaled hardly ever.
//
// A warp issues one cp.async of 512 gathered bytes in about 70 clocks, so the copies
// of a tile (64 of them) want several warps; in the scanning warps they made the scan
// the bottleneck (64 tokens over 8K: 132 us against 117), in the weight warps the
// weights (161 us), and a single gathering warp takes 4,600 clocks a tile (190 us).
//
// What bounds it now: 64 query rows, the weight warps (4,800 clocks a tile, of which
// their own work is about 4,100 and the wait for the scores the rest; the tensor pipe is
// at 9%), then the second pass (2,200 clocks a tile); 32 rows over long caches, the scan
// (2,800 clocks for 20 pages) and the fixed 14,000 clocks from the launch to the
// first weights and 6,000 of the join.  64 tokens for 2 sequences of 8K slots, 32
// heads, with the weights accumulated: 128 us (146 MB of HBM traffic: 1.1 TB/s; 116 with
// weights of one f16 in four e5m2 parts, which differed from fp32 weights by 9e-4); four
// tokens for 4 sequences of 64K slots, 64 / 8 heads: 37 us; a step of 32 and 64 query
// heads a head at 32K: 18 and 23 us.
#include <cooperative_groups.h>

#include "cache.cuh"

namespace cg = cooperative_groups;

namespace focus {
namespace {

constexpr int kTile = 128;             // keys of a tile
constexpr int kD = 128;
constexpr int kTileBytes = kTile * kD;
constexpr int kMaxCluster = kMaxClusterBlocks;
constexpr float kBelow = 4.f, kTop = 8.f;   // e4m3 ends at 448: weights start at 2^4 and stay below 2^8
// Sums are held times 2^kLift: s_max - ref lies within [4 - 120, 8 + 64], so a row's
// largest term within 2^-92 and 2^96, and a term is lost only below 2^-34 of it.
constexpr int kLift = 24;

template <int R, bool kMulti>
struct TcCfg {
  // Weight warps: four TMEM lane quadrants times kParts parts of the rows; then the
  // scan warps, those that gather, and the one that issues the products.
  static constexpr int kParts = R == 64 ? 4 : 2, kSoftWarps = 4 * kParts, kScanWarps = R == 64 ? 3 : 5, kGatherWarps = 4,
                       kGatherWarp = kSoftWarps + kScanWarps, kMmaWarp = kGatherWarp + kGatherWarps,
                       kThreads = (kMmaWarp + 1) * 32;
  static constexpr int kStages = 3;
  static constexpr int kAhead = R == 64 ? 8 : 16;              // pages a scan warp fetches group ids of at a time
  static constexpr int kListed = 4;                            // tiles listed ahead of the weights
  // A scan round: kSlots slots a lane, so kPages pages a warp; the list holds what a
  // round can add to a tile and the tiles listed.
  static constexpr int kSlots = R == 64 ? 4 : 8, kPages = kSlots / 2, kRound = kPages * kScanWarps;
  static constexpr int kList = R == 64 ? 1024 : 2048;          // entries of the block's list of kept slots
  static_assert(kList >= kRound * kPage + kListed * kTile && kStages < kListed, "list too short");
  static constexpr int kRowBytes = 128;                        // P's bytes of a key, per chunk of 32 rows
  static constexpr int kPBytes = kTile * 4 * R;
  static constexpr int kEntryBytes = kMulti ? 16 : 8;
  // byte offsets in dynamic shared memory
  static constexpr int kK = 0, kV = kK + kStages * kTileBytes, kQ = kV + kStages * kTileBytes, kP = kQ + 2 * R * kD,
                       kListAt = kP + 2 * kPBytes, kIds = kListAt + kList * kEntryBytes, kTable = kIds + 2 * kScanWarps * kAhead * kPage * 2,
                       kSmem = kTable + (kMulti ? kCacheTableGroups * 8 : 0) + 1024;   // + alignment
  // The partials' inbox lies over P: a block writes into another only when that one's
  // tiles are done.
  static constexpr int kInbox = kP;
  static_assert((R > kMaxCluster ? R : kMaxCluster) * kD * 4 <= 2 * kPBytes, "inbox does not fit");
  static constexpr int kCols = 8 * R;                          // TMEM: S twice, O
};

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// kind::f8f6f4, A and B e4m3, fp32 accumulate; M = 128.
constexpr uint32_t idesc_f8(int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
// D[tmem] (+)= A[smem] * B[smem], 32 steps of the inner dimension
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
      ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// Shared-memory descriptor of an operand with rows of 128 bytes; see sw128_desc.
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t lbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3fffu) | static_cast<uint64_t>((lbo >> 4) & 0x3fffu) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

// Arrives on `bar` (counted in its arrivals) when this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The e4m3 parts of two weights of at most 2^8: the first parts of both, then the second
// ones; and the third and fourth ones.  A part leaves at most 2^-4 of what it stands for
// (half a step of four bits), so sixteen times that fits the next one.  The rest behind
// the first part is held in f16, at most 2^-16 of the weight off; what follows is exact.
__device__ __forceinline__ void split_e4m3(float p0, float p1, uint32_t& c12, uint32_t& c34) {
  const uint32_t c1 = float2_to_e4m3x2(p0, p1);
  const float2 h = e4m3x2_to_float2(static_cast<uint16_t>(c1));
  float d0, d1;
  f2_unpack(f2_fma(f2_pack(h.x, h.y), f2_pack(-1.f, -1.f), f2_pack(p0, p1)), d0, d1);
  const __half2 sixteen = __floats2half2_rn(16.f, 16.f);
  __half2 r = __hmul2(__floats2half2_rn(d0, d1), sixteen);
  auto part = [&]() {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t*>(&r)));
    return static_cast<uint32_t>(c);
  };
  auto rest = [&](uint32_t c) {
    const uint32_t x = e4m3x2_to_f16x2(static_cast<uint16_t>(c));
    r = __hmul2(__hsub2(r, *reinterpret_cast<const __half2*>(&x)), sixteen);
  };
  const uint32_t c2 = part();
  rest(c2);
  const uint32_t c3 = part();
  rest(c3);
  c12 = c1 | c2 << 16;
  c34 = c3 | part() << 16;
}

// mbar_wait that reads the clock only after a few tries (the read costs as much as most
// of these waits).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) return true;
  return mbar_wait(bar, parity, abort, err);
}

__device__ __forceinline__ uint64_t bits_from(int k) {   // bits k ... 63
  return k >= 64 ? 0ull : ~0ull << max(k, 0);
}

template <int R, bool kMulti>
__global__ void __launch_bounds__(TcCfg<R, kMulti>::kThreads, 1)
    cache_attn_tc_kernel(CacheAttnLaunch L) {
  using C = TcCfg<R, kMulti>;
  constexpr int kStages = C::kStages, RH = R / C::kParts, kList = C::kList, kSlots = C::kSlots, kPages = C::kPages;
  constexpr int kRound = C::kRound, kLanes = kPage / kSlots;   // lanes a page
  constexpr int kParts = C::kParts, kSoftWarps = C::kSoftWarps, kMmaWarp = C::kMmaWarp, kThreads = C::kThreads,
                kScanWarps = C::kScanWarps, kGatherWarp = C::kGatherWarp, kGatherWarps = C::kGatherWarps, kListed = C::kListed, kAhead = C::kAhead;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t k_full[kStages], v_full[kStages], qk_done[kStages], pv_done[kStages], s_ready[2], p_ready[2];
  __shared__ uint64_t listed[kListed], used[kListed];  // a tile's entries are in the list; the weight warps have read them
  __shared__ uint64_t part_bar[kParts], soft_bar, scan_bar; // the four warps of a part; all weight warps; the scan's
  __shared__ uint2 s_found[2][kScanWarps];             // slots that a scan warp lists in a round, and its scales' range
  __shared__ int s_grow[kParts][3];                    // some reference of the part moves in this tile
  // Keys of a tile (by slot modulo 8), and kWide where the scales scanned by then lie more
  // than kScaleSpan apart; 0 ends a pass.
  __shared__ int s_cnt[8];
  constexpr int kWide = 256;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort_word;
  __shared__ __align__(16) float s_factor[R], s_minus[R], s_lse[R];   // the references and log2 sums, negated
  __shared__ int s_top[4][R];                          // per lane quadrant, in integer order
  __shared__ float s_l[4][R];
  __shared__ float s_w[2][kParts][kTile];              // slots' weights by part (pass 1)
  float (*s_weight)[R] = reinterpret_cast<float (*)[R]>(&s_w[0][0][0]);   // weight of a block's partial in a row (join)
  static_assert(sizeof(s_w) >= kMaxCluster * R * sizeof(float), "shared");
  __shared__ float2 s_all[kMaxCluster][R];             // the cluster's references and sums
  __shared__ uint32_t s_nan[kMulti ? R : 1][4];        // outputs that a kept NaN value reaches
  volatile int* abort = &s_abort_word;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  int4* list4 = reinterpret_cast<int4*>(smem + C::kListAt);
  int2* list2 = reinterpret_cast<int2*>(smem + C::kListAt);
  float* inbox = reinterpret_cast<float*>(smem + C::kInbox);
  unsigned long long* table = reinterpret_cast<unsigned long long*>(smem + C::kTable);   // rows per group id
  cg::cluster_group cluster = cg::this_cluster();
  const int h = blockIdx.y, b = blockIdx.z, cs = gridDim.x, rank = blockIdx.x;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = L.H / L.H_kv;
  const int n = cache_len(L.c, L.H_kv, b, h, L.err);
  const int fresh = cache_new(L.n_new, L.n, b, L.err);
  const int pos0 = L.c.next[b] - fresh;                // position of token 0
  const int rows = G * fresh;
  const int pages = (n + kPage - 1) / kPage;
  const int near_from = n - static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(L.w) + fresh));
  const int32_t* gids = L.gid + (static_cast<size_t>(b) * L.A + (L.A == 1 ? 0 : h)) * L.n;

  if (threadIdx.x == 0) {
    s_abort_word = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&k_full[i], kGatherWarps * 32);
      mbar_init(&v_full[i], kGatherWarps * 32);
      mbar_init(&qk_done[i], 1);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < kListed; ++i) {
      mbar_init(&listed[i], kScanWarps);
      mbar_init(&used[i], kSoftWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_ready[i], 1);
      mbar_init(&p_ready[i], kSoftWarps);
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&part_bar[i], 4);
      s_grow[i][0] = s_grow[i][1] = s_grow[i][2] = 0;
    }
    mbar_init(&soft_bar, kSoftWarps);
    mbar_init(&scan_bar, kScanWarps);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&s_tmem, C::kCols);
  // rows of a partial tile that no gather fills meet weights of 0: they must not be NaN
  for (int i = threadIdx.x; i < kStages * kTileBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + C::kV)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t tmem_o = tmem + 4 * R;
  uint32_t part_phase = 0, soft_phase = 0, scan_phase = 0;   // uses of the barriers so far
  // Bounded barrier among the warps that share `bar` (a plain named barrier would
  // wait for ever on a warp that gave up).
  auto meet = [&](uint64_t* bar, uint32_t& phase) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    wait(bar, phase++ & 1, abort, L.err);
  };
  uint32_t it = 0;                                     // slots (tiles and end marks) so far, the same in every role
  uint32_t skip = 0;                                   // of them in second passes, which use no values: V's slot is it - skip

  for (int r0 = 0; r0 < rows; r0 += R) {
    const int t_lo = r0 / G, off = r0 - t_lo * G;      // the block's rows start `off` rows into token t_lo
    const int live = min(R, rows - r0);
    const int tokens = (r0 + live - 1) / G - t_lo + 1;
    const int gid0 = gids[t_lo];
    // ---- the scan's state, and its first loads.  Pages rank, rank + cs, ... in rounds of
    // kRound, kPages a warp: its page x is number x / kPages * kRound + v * kPages +
    // x % kPages of them.
    const int v = warp - kSoftWarps;
    auto page_of = [&](int x) { return rank + (x / kPages * kRound + v * kPages + x % kPages) * cs; };
    auto entry_of = [&](int x) {                   // table entry of the warp's page x + lane, unchecked
      const int j = page_of(x + lane);
      return lane < kAhead && j < L.c.max_pages ? L.c.table[static_cast<size_t>(b) * L.c.max_pages + j] : -1;
    };
    uint8_t* ids = smem + C::kIds + v * 2 * kAhead * kPage * 2;      // two batches of kAhead pages
    int next_page = -1, lane_page = -1, lane_exps = 0, entry = 0;
    // Value exponents of the pages begun: the largest + 64 and 120 - the smallest in two
    // 16-bit halves, of this warp and of all scan warps.
    uint32_t my_range = 0, range = 0;
    auto wide = [&]() { return static_cast<int>((range & 0xffffu) + (range >> 16)) - (kMaxExp - kMinExp) > kScaleSpan; };
    PageScales next_scales{1.f, 1.f};
    auto fetch = [&](int x) {                      // starts on pages x ... x + kAhead - 1, and on the table behind them
      next_page = -1;
      if (lane < kAhead && page_of(x + lane) < pages) {
        next_page = entry;
        if (entry < 0 || entry >= L.c.n_pages) {
          atomicOr(L.err, kErrBadCache);
          next_page = -1;
        }
      }
      __syncwarp();
#pragma unroll
      for (int y = 0; y < kAhead * kPage * 2 / 16 / 32; ++y) {
        const int page = __shfl_sync(~0u, next_page, y * 4 + lane / 8);
        if (page >= 0)
          cp_async_16(ids + (x / kAhead & 1) * kAhead * kPage * 2 + y * 512 + lane * 16,
                      L.c.gid + (static_cast<size_t>(page) * L.H_kv + h) * kPage + lane % 8 * 8, 16);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (next_page >= 0) next_scales.load(L.c, static_cast<size_t>(next_page) * L.H_kv + h);
      entry = entry_of(x + kAhead);
    };
    const bool scans = warp >= kSoftWarps && warp < kGatherWarp;
    if (scans) {
      entry = entry_of(0);
      fetch(0);
    }
    // ---- queries: two e4m3 parts, a warp a row; references, masks
    if (warp < kSoftWarps) {
      uint2 u[R / kSoftWarps];
#pragma unroll
      for (int i = 0; i < R / kSoftWarps; ++i) {
        const int r = warp + i * kSoftWarps, g = (r0 + r) % G, t = (r0 + r) / G;
        u[i] = make_uint2(0, 0);
        if (r < live)
          u[i] = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(L.Q) +
                                                ((static_cast<size_t>(b) * L.H + h * G + g) * L.n + t) * kD)[lane];
      }
#pragma unroll
      for (int i = 0; i < R / kSoftWarps; ++i) {
        const int r = warp + i * kSoftWarps;
        const float f[4] = {__uint_as_float(u[i].x << 16), __uint_as_float(u[i].x & 0xffff0000u),
                            __uint_as_float(u[i].y << 16), __uint_as_float(u[i].y & 0xffff0000u)};
        uint32_t top = 0;
        bool finite = true;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a = __float_as_uint(f[e]) & 0x7fffffffu;
          if (a < 0x7f800000u) top = max(top, a);
          else finite = false;
        }
        top = __reduce_max_sync(~0u, top);
        finite = __all_sync(~0u, finite);
        const int eq = need_exp(top, kMinQueryExp);
        const float down = exp2_int(-eq);
        uint32_t part[2];
        const uint16_t a = float2_to_e4m3x2(f[0] * down, f[1] * down), c = float2_to_e4m3x2(f[2] * down, f[3] * down);
        const float2 fa = e4m3x2_to_float2(a), fc = e4m3x2_to_float2(c);
        part[0] = a | static_cast<uint32_t>(c) << 16;
        part[1] = float2_to_e4m3x2((f[0] * down - fa.x) * 16.f, (f[1] * down - fa.y) * 16.f) |
                  static_cast<uint32_t>(float2_to_e4m3x2((f[2] * down - fc.x) * 16.f, (f[3] * down - fc.y) * 16.f)) << 16;
#pragma unroll
        for (int p = 0; p < 2; ++p)
          *reinterpret_cast<uint32_t*>(smem + C::kQ + (p * R + r) * kD + ((lane / 4) ^ (r & 7)) * 16 + lane % 4 * 4) = part[p];
        if (lane == 0) {
          // rows with an infinite or NaN element become NaN through their factor
          s_factor[r] = finite ? exp2_int(eq) * L.scale_log2 : __int_as_float(0x7fffffff);
          s_minus[r] = -kNoRef;
        }
      }
      fence_proxy_async_smem();
    }
    if (kMulti) {
      for (int i = threadIdx.x; i < kCacheTableGroups; i += kThreads) table[i] = 0;
      for (int i = threadIdx.x; i < R * 4; i += kThreads) s_nan[i / 4][i % 4] = 0;
      __syncthreads();
      if (threadIdx.x < tokens) {
        const int g = gids[t_lo + threadIdx.x];
        const uint64_t mine = bits_from(threadIdx.x * G - off) & ~bits_from((threadIdx.x + 1) * G - off) & ~bits_from(live);
        if (g >= 0 && g < kCacheTableGroups) atomicOr(&table[g], mine);
      }
    }
    __syncthreads();

    int entries = 0, tiles = 0;                        // load warp: listed slots; softmax warps: tiles of pass 0
    for (int pass = 0; pass < (L.accumulate ? 2 : 1); ++pass) {
      const uint32_t it0 = it;
      if (scans) {
        // ------------------------------------------------ scan
        const bool relist = pass == 0 || entries > kList;  // else the whole list is still there
        int x = 0;                                     // the warp's next page
        if (relist) entries = 0;
        auto scan_round = [&]() {
          if (x % kAhead == 0) {                       // a new batch: it becomes current, the next one is fetched
            lane_page = next_page;
            lane_exps = next_scales.bytes();
            const int ve = static_cast<int8_t>(lane_exps >> 8);
            const uint32_t high = __reduce_max_sync(~0u, lane_page >= 0 ? static_cast<uint32_t>(ve - kMinExp) : 0u);
            const uint32_t low = __reduce_max_sync(~0u, lane_page >= 0 ? static_cast<uint32_t>(kMaxExp - ve) : 0u);
            my_range = __vmaxu2(my_range, high | low << 16);
            fetch(x + kAhead);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
          }
          const int sub = lane / kLanes, at_page = x % kAhead + sub, slot0 = lane % kLanes * kSlots;
          const int page = __shfl_sync(~0u, lane_page, at_page), exps = __shfl_sync(~0u, lane_exps, at_page);
          const int j = page_of(x + sub), s = j * kPage + slot0;
          uint32_t idw[kSlots / 2];
          const uint2* src = reinterpret_cast<const uint2*>(ids + (x / kAhead & 1) * kAhead * kPage * 2 +
                                                            (at_page * kPage + slot0) * 2);
#pragma unroll
          for (int e = 0; e < kSlots / 4; ++e) {
            idw[2 * e] = src[e].x;
            idw[2 * e + 1] = src[e].y;
          }
          const size_t plane = static_cast<size_t>(max(page, 0)) * L.H_kv + h;
          const int left = page >= 0 ? n - s : 0;      // slots of this lane that are in use
          uint64_t mk[kSlots];                         // rows that keep the slot
          uint32_t kept = 0;
#pragma unroll
          for (int e = 0; e < kSlots; ++e) {
            const int id = static_cast<int16_t>(idw[e / 2] >> (e % 2 * 16));
            if (kMulti) mk[e] = id >= 0 && id < kCacheTableGroups ? table[id] : 0ull;
            else mk[e] = id == gid0;
          }
          const bool near = page >= 0 && (j + 1) * kPage > near_from;
          if (__any_sync(~0u, near)) {
            int at[kSlots];
#pragma unroll
            for (int e = 0; e < kSlots; e += 4) {
              int4 p = make_int4(0, 0, 0, 0);
              if (near) p = *reinterpret_cast<const int4*>(L.c.pos + plane * kPage + slot0 + e);
              at[e] = p.x; at[e + 1] = p.y; at[e + 2] = p.z; at[e + 3] = p.w;
            }
#pragma unroll
            for (int e = 0; e < kSlots; ++e) {
              if (!near) continue;
              if (kMulti) {
                // tokens from `from` on are not before the slot, those before `to` have it in their window
                const long long ahead = static_cast<long long>(at[e]) - pos0 - t_lo;
                const int from = static_cast<int>(min(max(ahead, 0ll), static_cast<long long>(tokens)));
                const int to = static_cast<int>(min(max(ahead + L.w, 0ll), static_cast<long long>(tokens)));
                const uint64_t after = bits_from(from * G - (from ? off : 0)) & ~bits_from(live);
                mk[e] = (mk[e] & after) | (after & ~bits_from(to * G - (to ? off : 0)));
              } else {
                mk[e] = cache_keep(pos0, at[e], L.w, mk[e] != 0);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < kSlots; ++e)
            if (e < left && mk[e]) kept |= 1u << e;
          // ranks: lanes of the warp, then the warps of the round
          int sum = __popc(kept);
          const int mine = sum;
#pragma unroll
          for (int y = 1; y < 32; y *= 2) {
            const int u = __shfl_up_sync(~0u, sum, y);
            if (lane >= y) sum += u;
          }
          const int turn = x / kPages & 1;
          if (lane == 31) s_found[turn][v] = make_uint2(sum, my_range);
          meet(&scan_bar, scan_phase);
          int at = entries + sum - mine;
#pragma unroll
          for (int w = 0; w < kScanWarps; ++w) {
            const uint2 word = s_found[turn][w];
            const int found = word.x;
            range = __vmaxu2(range, word.y);
            if (w < v) at += found;
            entries += found;
          }
          const uint32_t row = static_cast<uint32_t>(plane) * kPage + slot0;
#pragma unroll
          for (int e = 0; e < kSlots; ++e)
            if (kept >> e & 1) {
              if (kMulti)
                list4[at & (kList - 1)] = make_int4(row + e, exps, static_cast<int>(mk[e]), static_cast<int>(mk[e] >> 32));
              else
                list2[at & (kList - 1)] = make_int2(row + e, exps);
              ++at;
            }
          x += kPages;
        };
        // the round's first page lies behind the end (the same in all scan warps)
        auto scanned = [&]() { return !relist || rank + x / kPages * kRound * cs >= pages; };
        for (int tile = 0;; ++tile, ++it) {
          if (it >= kListed) wait(&used[it % kListed], (it / kListed + 1) & 1, abort, L.err);
          while (entries < (tile + 1) * kTile && !scanned()) scan_round();
          const int cnt = max(min(kTile, entries - tile * kTile), 0);
          if (v == 0 && lane == 0) s_cnt[it & 7] = cnt > 0 && wide() ? cnt | kWide : cnt;
          __syncwarp();
          if (lane == 0) mbar_arrive(&listed[it % kListed]);       // with every warp's: the tile's entries are there
          if (cnt == 0 || *abort) {
            ++it;
            break;
          }
        }
        cp_async_wait_all();
        if (pass == 0 && L.accumulate && entries > kList) {        // the second pass starts over
          entry = entry_of(0);
          fetch(0);
        }
      } else if (warp >= kGatherWarp && warp < kMmaWarp) {
        // ------------------------------------------------ gathers of kept rows
        // Four rows a step and warp (a step is a multiple of 8 rows on: one swizzle for
        // all).  K's stage is free once its products are done, V's once the weights' are.
        constexpr int kStep = 4 * kGatherWarps, kSteps = kTile / kStep;
        static_assert(kStep % 8 == 0, "swizzle");
        const int row0 = (warp - kGatherWarp) * 4 + lane / 8;
        const uint32_t to_row = row0 * kD + (lane % 8 ^ (row0 & 7)) * 16, piece = lane % 8 * 16;
        for (int tile = 0;; ++tile, ++it) {
          const int st = it % kStages;
          const uint32_t parity = (it / kStages + 1) & 1;
          const bool ok = __all_sync(~0u, wait(&listed[it % kListed], (it / kListed) & 1, abort, L.err));
          const int cnt = ok ? s_cnt[it & 7] & (kWide - 1) : 0;
          const int base = (tile * kTile & (kList - 1)) + row0;
          uint32_t from[kSteps];
#pragma unroll
          for (int y = 0; y < kSteps; ++y)
            from[y] = row0 + y * kStep < cnt ? static_cast<uint32_t>(kMulti ? list4[base + y * kStep].x : list2[base + y * kStep].x) : 0u;
          auto copy = [&](uint8_t* to, const uint8_t* pool) {
#pragma unroll
            for (int y = 0; y < kSteps; ++y)
              if (row0 + y * kStep < cnt)
                cp_async_16(to + to_row + y * kStep * kD, pool + static_cast<size_t>(from[y]) * kD + piece, 16);
          };
          if (it >= kStages) wait(&qk_done[st], parity, abort, L.err);
          if (cnt > 0) {
            copy(smem + C::kK + st * kTileBytes, L.c.k);
            cp_async_arrive(&k_full[st]);
          } else {
            mbar_arrive(&k_full[st]);
          }
          if (pass == 0) {
            const uint32_t vi = it - skip;
            if (vi >= kStages) wait(&pv_done[vi % kStages], (vi / kStages + 1) & 1, abort, L.err);
            if (cnt > 0) {
              copy(smem + C::kV + vi % kStages * kTileBytes, L.c.v);
              cp_async_arrive(&v_full[vi % kStages]);
            } else {
              mbar_arrive(&v_full[vi % kStages]);
            }
          }
          if (cnt == 0 || *abort) {
            ++it;
            break;
          }
        }
        cp_async_wait_all();
      } else if (warp == kMmaWarp) {
        // ------------------------------------------------ products
        if (lane == 0) {
          const uint32_t kb = smem_u32(smem + C::kK), vb = smem_u32(smem + C::kV), qb = smem_u32(smem + C::kQ),
                         pb = smem_u32(smem + C::kP);
          bool ok = true;
          auto scores = [&](uint32_t slot) {           // S of a slot whose K is there; false at the end of the pass
            const int st = slot % kStages;
            if (!ok || s_cnt[slot & 7] == 0) {
              mbar_arrive(&qk_done[st]);
              mbar_arrive(&s_ready[slot & 1]);
              return false;
            }
            fence_proxy_async_smem();                  // the copies, like all writes of threads, to the tensor core
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < kD / 32; ++x)
              mma_f8(tmem + (slot & 1) * 2 * R, desc_rows(kb + st * kTileBytes + x * 32, 16),
                     desc_rows(qb + x * 32, 16), idesc_f8(2 * R, false, false), x > 0);
            mma_commit(&qk_done[st]);
            mma_commit(&s_ready[slot & 1]);
            return true;
          };
          auto k_wait = [&](uint32_t slot) {
            ok = ok && mbar_wait_nap(&k_full[slot % kStages], (slot / kStages) & 1, abort, L.err);
            ok = ok && mbar_wait(&listed[slot % kListed], (slot / kListed) & 1, abort, L.err);     // done: orders s_cnt
          };
          k_wait(it);
          bool have = scores(it);
          bool first = true;
          while (have) {
            const uint32_t vi = it - skip;
            const int st = vi % kStages;
            const int cnt = s_cnt[it & 7] & (kWide - 1);
            // The next tile's S if its K comes before this tile's P (its S buffer was read
            // before P of slot it - 1 was ready); else after this tile's product.
            bool next = false, asked = false;
            const unsigned long long since = global_ns();
            while (ok && !asked && !mbar_test_wait(&p_ready[it & 1], (it >> 1) & 1)) {
              if (mbar_test_wait(&k_full[(it + 1) % kStages], ((it + 1) / kStages) & 1)) {
                k_wait(it + 1);
                next = scores(it + 1);
                asked = true;
              } else {
                __nanosleep(kNapNs);
                if (*abort || global_ns() - since > kWaitTimeoutNs) ok = false;   // the wait below reports it
              }
            }
            ok = mbar_wait_nap(&p_ready[it & 1], (it >> 1) & 1, abort, L.err) && ok;
            if (pass == 0) ok = ok && mbar_wait_nap(&v_full[st], (vi / kStages) & 1, abort, L.err);
            if (pass == 0 && ok) {
              fence_proxy_async_smem();
              tc_fence_after();
              for (int x = 0; x < (cnt + 31) / 32; ++x)
                mma_f8(tmem_o, desc_rows(vb + st * kTileBytes + x * 32 * kD, 16),
                       desc_rows(pb + (it & 1) * C::kPBytes + x * 32 * C::kRowBytes, kTile * C::kRowBytes),
                       idesc_f8(4 * R, true, true), !(first && x == 0));
            }
            if (pass == 0) mma_commit(&pv_done[st]);
            first = false;
            if (!asked) {
              k_wait(it + 1);
              next = scores(it + 1);
            }
            have = next && ok;
            ++it;
          }
          // Every commit has arrived before the block ends.  The end mark's V slot is passed on
          // once the gathering warps have seen the stage's last one.
          if (!first) mbar_wait(&qk_done[(it - 1) % kStages], ((it - 1) / kStages) & 1, abort, L.err);
          if (pass == 0) {
            const uint32_t vi = it - skip;
            if (!first) mbar_wait(&pv_done[(vi - 1) % kStages], ((vi - 1) / kStages) & 1, abort, L.err);
            mbar_wait_nap(&v_full[vi % kStages], (vi / kStages) & 1, abort, L.err);
            mbar_arrive(&pv_done[vi % kStages]);
          }
          ++it;
        }
        it = __shfl_sync(~0u, it, 0);
      } else {
        // ------------------------------------------------ weights: one key a thread, a part of the rows
        const int quad = warp & 3, part = warp >> 2, key = quad * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        uint64_t l2[RH / 2];                           // row sums, in pairs
#pragma unroll
        for (int r = 0; r < RH / 2; ++r) l2[r] = f2_pack(0.f, 0.f);
        int tile = 0;
        for (;; ++tile, ++it) {
          const uint32_t vi = it - skip;
          const int st = vi % kStages, buf = it & 1;
          const bool ok = wait(&s_ready[buf], (it >> 1) & 1, abort, L.err);
          const int tile_word = ok ? s_cnt[it & 7] : 0, cnt = tile_word & (kWide - 1);
          if (__any_sync(~0u, cnt == 0)) {
            if (lane == 0) {
              mbar_arrive(&p_ready[buf]);
              mbar_arrive(&used[it % kListed]);
            }
            ++it;
            break;
          }
          tc_fence_after();
          int ex, mask;
          uint32_t pool_row;
          {
            const int idx = (tile * kTile + key) & (kList - 1);
            if (kMulti) {
              const int4 e = list4[idx];
              pool_row = e.x;
              ex = e.y;
              mask = static_cast<int>(static_cast<uint32_t>(part * RH < 32 ? e.z : e.w) >> (part * RH % 32));
            } else {
              const int2 e = list2[idx];
              pool_row = e.x;
              ex = e.y;
              mask = static_cast<int>(~static_cast<uint32_t>(bits_from(live - part * RH)));
            }
            if (key >= cnt) mask = ex = 0;
          }
          const float kf = exp2_int(static_cast<int8_t>(ex)), ve = static_cast<float>(static_cast<int8_t>(ex >> 8));
          uint32_t hi[RH], lo[RH];
          tmem_ld(tmem + lanes + buf * 2 * R + part * RH, hi);
          tmem_ld(tmem + lanes + buf * 2 * R + R + part * RH, lo);
          tmem_wait_ld();
          if (pass == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[buf]);
            float w = 0.f, w1 = 0.f;
            const uint64_t sixteenth = f2_pack(0.0625f, 0.0625f), kf2 = f2_pack(kf, kf);
#pragma unroll
            for (int r = 0; r < RH; r += 4) {
              uint64_t f01, f23, m01, m23;
              lds_f2x2(&s_factor[part * RH + r], f01, f23);
              lds_f2x2(&s_lse[part * RH + r], m01, m23);
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const uint64_t h2 = f2_pack(__uint_as_float(hi[r + e]), __uint_as_float(hi[r + e + 1]));
                const uint64_t l2 = f2_pack(__uint_as_float(lo[r + e]), __uint_as_float(lo[r + e + 1]));
                float d0, d1;
                f2_unpack(f2_fma(f2_mul(f2_fma(l2, sixteenth, h2), e ? f23 : f01), kf2, e ? m23 : m01), d0, d1);
                const float p0 = exp2_fast(d0), p1 = exp2_fast(d1);
                w += mask >> (r + e) & 1 ? p0 : 0.f;
                w1 += mask >> (r + e + 1) & 1 ? p1 : 0.f;
              }
            }
            w += w1;
            if (part) s_w[buf][part][key] = w;
            meet(&soft_bar, soft_phase);
            if (lane == 0) mbar_arrive(&used[it % kListed]);
            if (!part && key < cnt) {
              for (int x = 1; x < kParts; ++x) w += s_w[buf][x][key];
              atomicAdd(L.c.mass + pool_row, w);       // the only addition to this slot for these rows: its order cannot matter
            }
            continue;
          }
          // t = s 2^(e_k) + e_v, two rows a step
          float t[RH], over = -INFINITY;
          const uint64_t sixteenth = f2_pack(0.0625f, 0.0625f), kf2 = f2_pack(kf, kf), ve2 = f2_pack(ve, ve);
#pragma unroll
          for (int r = 0; r < RH; r += 4) {
            uint64_t f01, f23, m01, m23;
            lds_f2x2(&s_factor[part * RH + r], f01, f23);
            lds_f2x2(&s_minus[part * RH + r], m01, m23);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const uint64_t h2 = f2_pack(__uint_as_float(hi[r + e]), __uint_as_float(hi[r + e + 1]));
              const uint64_t l2 = f2_pack(__uint_as_float(lo[r + e]), __uint_as_float(lo[r + e + 1]));
              const uint64_t t2 = f2_fma(f2_mul(f2_fma(l2, sixteenth, h2), e ? f23 : f01), kf2, ve2);
              float t0, t1, d0, d1;
              f2_unpack(t2, t0, t1);
              if (!(mask >> (r + e) & 1)) t0 = -INFINITY;
              if (!(mask >> (r + e + 1) & 1)) t1 = -INFINITY;
              f2_unpack(f2_add(f2_pack(t0, t1), e ? m23 : m01), d0, d1);
              t[r + e] = t0;
              t[r + e + 1] = t1;
              over = fmaxf(over, fmaxf(d0, d1));
            }
          }
          // (three flags in turn: the one cleared here was last read before the previous meeting)
          if (quad == 0 && lane == 0) s_grow[part][(it + 1) % 3] = 0;
          if (__any_sync(~0u, over > kTop) && lane == 0) s_grow[part][it % 3] = 1;
          meet(&part_bar[part], part_phase);
          if (s_grow[part][it % 3]) {
            // some row's reference moves, by the row's own weights: rows do not touch each
            // other.  Lane r takes row r (the same result in the part's four warps).
            int top = INT_MIN;
#pragma unroll
            for (int r = 0; r < RH; ++r) {
              const int u = __float_as_int(t[r]), order = u ^ (u >> 31 & 0x7fffffff);   // floats' order as integers
              const int m = __reduce_max_sync(~0u, t[r] == t[r] ? order : INT_MIN);
              if (lane == r) top = m;
            }
            if (lane < RH) s_top[quad][part * RH + lane] = top;
            meet(&part_bar[part], part_phase);
            float moved = 0.f, fh = 1.f;               // the factor's root: it may lie below the normals where sums do not
            if (lane < RH) {
              const int rr = part * RH + lane;
              const int m = max(max(s_top[0][rr], s_top[1][rr]), max(s_top[2][rr], s_top[3][rr]));
              const float was = -s_minus[rr], highest = __int_as_float(m ^ (m >> 31 & 0x7fffffff));
              moved = highest > was + kTop ? highest - kBelow : was;
              fh = exp2_fast(0.5f * (was - moved));
            }
#pragma unroll
            for (int r = 0; r < RH; r += 2) {
              const uint64_t fh2 = f2_pack(__shfl_sync(~0u, fh, r), __shfl_sync(~0u, fh, r + 1));
              l2[r / 2] = f2_mul(f2_mul(l2[r / 2], fh2), fh2);
            }
            if (tile > 0) {
              mbar_wait(&pv_done[(vi - 1) % kStages], ((vi - 1) / kStages) & 1, abort, L.err);
              tc_fence_after();
#pragma unroll
              for (int y = 0; y < RH / 2; ++y) {       // two rows, eight columns
                float f0 = __shfl_sync(~0u, fh, 2 * y), f1 = __shfl_sync(~0u, fh, 2 * y + 1);
                if (f0 == 1.f && f1 == 1.f) continue;
                f0 *= f0;
                f1 *= f1;
                uint32_t v[8];
                tmem_ld(tmem_o + lanes + part * 4 * RH + y * 8, v);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * (x & 1 ? f1 : f0));
                tmem_st8(tmem_o + lanes + part * 4 * RH + y * 8, v);
              }
              tmem_wait_st();
            }
            meet(&part_bar[part], part_phase);         // every warp has read the old references
            if (quad == 0 && lane < RH) s_minus[part * RH + lane] = -moved;
            meet(&part_bar[part], part_phase);
          }
          if (tile > 1)                                // P of the slot before the last one has been used
            wait(&pv_done[(vi - 2) % kStages], ((vi - 2) / kStages) & 1, abort, L.err);
          float vf = exp2_int(kLift - static_cast<int8_t>(ex >> 8));
          if (tile_word & kWide) {                     // the sum's terms on their own (the same in all warps)
            const float up = static_cast<float>(kLift) - ve;
#pragma unroll
            for (int r = 0; r < RH; r += 2) {
              const float t0 = t[r] + s_minus[part * RH + r] + up, t1 = t[r + 1] + s_minus[part * RH + r + 1] + up;
              l2[r / 2] = f2_add(l2[r / 2], f2_pack(exp2_fast(t0), exp2_fast(t1)));
            }
            vf = 0.f;
          }
          const uint64_t vf2 = f2_pack(vf, vf);
          uint32_t word[RH];
#pragma unroll
          for (int r = 0; r < RH; r += 4) {
            uint64_t m01, m23;
            lds_f2x2(&s_minus[part * RH + r], m01, m23);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              float d0, d1;
              f2_unpack(f2_add(f2_pack(t[r + e], t[r + e + 1]), e ? m23 : m01), d0, d1);
              const float p0 = exp2_fast(d0), p1 = exp2_fast(d1);
              l2[(r + e) / 2] = f2_fma(f2_pack(p0, p1), vf2, l2[(r + e) / 2]);
              split_e4m3(p0, p1, word[r + e], word[r + e + 1]);
            }
          }
          // this thread's 4 RH bytes of the key's row of P (R = 64: two chunks of 128 bytes)
          constexpr int kPieces = RH / 4, kInRow = C::kRowBytes / 16;
          uint8_t* prow = smem + C::kP + buf * C::kPBytes + part * kPieces / kInRow * kTile * C::kRowBytes + key * C::kRowBytes;
#pragma unroll
          for (int c = 0; c < kPieces; ++c)
            *reinterpret_cast<uint4*>(prow + ((part * kPieces % kInRow + c) ^ (key & 7)) * 16) =
                make_uint4(word[4 * c], word[4 * c + 1], word[4 * c + 2], word[4 * c + 3]);
          if (kMulti) {
            // A row that does not keep a key has weight 0 for it, and 0 * NaN would reach
            // that row: NaN codes leave the tile and mark the outputs that they reach.
            wait(&v_full[st], (vi / kStages) & 1, abort, L.err);
            uint32_t any = 0;
            uint4* vrow = reinterpret_cast<uint4*>(smem + C::kV + st * kTileBytes + key * kD);
#pragma unroll
            for (int c = 0; c < 8 / kParts; ++c) {
              const uint4 u = vrow[(part * (8 / kParts) + c) ^ (key & 7)];
              const uint32_t m = 0x7f7f7f7fu, one = 0x01010101u;       // a magnitude of 127 carries into the sign's bit
              any |= ((u.x & m) + one) | ((u.y & m) + one);
              any |= ((u.z & m) + one) | ((u.w & m) + one);
            }
            if (any & 0x80808080u) {
              uint8_t* bytes = reinterpret_cast<uint8_t*>(vrow);
              const int4 e = list4[(tile * kTile + key) & (kList - 1)];
              const uint64_t keepers = key < cnt ? static_cast<uint32_t>(e.z) | static_cast<uint64_t>(static_cast<uint32_t>(e.w)) << 32 : 0ull;
              for (int d = part * (kD / kParts); d < (part + 1) * (kD / kParts); ++d) {
                uint8_t* at = bytes + ((d / 16) ^ (key & 7)) * 16 + d % 16;
                if ((*at & 127) != 127) continue;
                *at = 0;
                for (int r = 0; r < R; ++r)
                  if (keepers >> r & 1) atomicOr(&s_nan[r][d / 32], 1u << (d % 32));
              }
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&p_ready[buf]);
            mbar_arrive(&used[it % kListed]);
          }
        }
        if (pass == 0) {
          // ---- the block's partial: every row's sum, and its part of O to the block that writes it
          tiles = tile;
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            float l0, l1;
            f2_unpack(l2[r / 2], l0, l1);
            float x = r & 1 ? l1 : l0;
#pragma unroll
            for (int y = 16; y > 0; y /= 2) x += __shfl_xor_sync(~0u, x, y);
            if (lane == 0) s_l[quad][part * RH + r] = x;
          }
          if (tiles > 0) {
            const uint32_t last = it - skip - 2;       // the last tile's slot: `it` is past the end mark
            mbar_wait(&pv_done[last % kStages], (last / kStages) & 1, abort, L.err);
            tc_fence_after();
          }
        }
      }
      __syncwarp();
      if (pass == 1) {
        skip += it - it0;
        break;
      }

      // ---- join: the same exchange as in cache_attn.cu
      cluster.sync();                                  // every block runs and is past its last round
      const int share = (R + cs - 1) / cs;             // rows that a block writes
      if (warp < kSoftWarps) {
        const int quad = warp & 3, part = warp >> 2, d = quad * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        if (tiles > 0) {
#pragma unroll
          for (int y = 0; y < RH / 2; ++y) {           // two rows: part 1 of both, then parts 2, 3, 4
            uint32_t v[8];
            tmem_ld(tmem_o + lanes + part * 4 * RH + y * 8, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = part * RH + 2 * y + e;
              float x = fmaf(fmaf(fmaf(__uint_as_float(v[6 + e]), 0.0625f, __uint_as_float(v[4 + e])), 0.0625f,
                                  __uint_as_float(v[2 + e])), 0.0625f, __uint_as_float(v[e]));
              if (kMulti && (s_nan[kMulti ? r : 0][quad] >> lane & 1)) x = __int_as_float(0x7fffffff);
              const int to = r / share;
              *cluster.map_shared_rank(inbox + (rank * share + r - to * share) * kD + d, to) = x;
            }
          }
        }
      }
      for (int i = threadIdx.x; i < R * cs; i += kThreads) {
        const int r = i % R, to = i / R;
        *cluster.map_shared_rank(&s_all[rank][r], to) =
            make_float2(-s_minus[r], (s_l[0][r] + s_l[1][r]) + (s_l[2][r] + s_l[3][r]));
      }
      tc_fence_before();
      cluster.sync();
      tc_fence_after();
      if (threadIdx.x < R) {
        const int r = threadIdx.x;
        float M = kNoRef, l = 0.f;
        for (int x = 0; x < cs; ++x) M = fmaxf(M, s_all[x][r].x);
        for (int x = 0; x < cs; ++x)
          if (s_all[x][r].y != 0.f) {
            const float fh = exp2f(0.5f * (s_all[x][r].x - M));
            l += s_all[x][r].y * fh * fh;
          }
        const float lse = l != 0.f ? M + (log2f(l) - kLift) : -INFINITY;
        s_lse[r] = l != 0.f ? -lse : kNoRef;
        for (int x = 0; x < cs; ++x)
          s_weight[x][r] = s_all[x][r].y != 0.f ? exp2f(s_all[x][r].x - M) / l * exp2_int(kLift) : 0.f;
        if (rank == 0 && L.lse && r < live)
          L.lse[(static_cast<size_t>(b) * L.H + h * G + (r0 + r) % G) * L.n + (r0 + r) / G] = lse * 0.6931471805599453f;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < share * (kD / 4); i += kThreads) {
        const int local = i / (kD / 4), r = rank * share + local, d = i % (kD / 4) * 4;
        if (r >= live) break;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int x = 0; x < cs; ++x) {
          if (s_all[x][r].y == 0.f) continue;          // nothing kept there
          const float f = s_weight[x][r];
          const float4 u = *reinterpret_cast<const float4*>(inbox + (x * share + local) * kD + d);
          a.x += u.x * f; a.y += u.y * f; a.z += u.z * f; a.w += u.w * f;
        }
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(L.O) +
                                  ((static_cast<size_t>(b) * L.H + h * G + (r0 + r) % G) * L.n + (r0 + r) / G) * kD + d) =
            make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
      }
      __syncthreads();
    }
    __syncthreads();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int R, bool kMulti>
ClusterFits g_fits;

template <int R, bool kMulti>
cudaError_t launch(const CacheAttnLaunch& L, cudaStream_t st) {
  // Blocks per (sequence, head): one wave of the clusters that run at once, as long as
  // each block scans a round or so.  Two in several waves where a block still has 64 pages
  // for each wave, 32 if there are several tokens, which keep more of a page.  (Four would
  // gain a fifth for several tokens in full tables of 512 pages, but sequences that fill
  // an eighth of theirs would lose half.)  Up to n pages for each of B sequences of 8 heads, us with 1, 2,
  // 4 blocks; * is taken:
  //   24 rows of one token   B = 8, n = 512: 62, 37*, 42     B = 16, n = 128: 41*, 43, 63
  //     B = 16, n = 256: 67, 42*, 67    B = 20, n = 256: 66*, 64, 86   n = 512: 136, 102*, 114
  //     B = 32, n = 256: 84*, 88, 130   n = 512: 145, 122*, 150        n = 1024: 277, 220*, 225
  //   32 rows of four tokens B = 8, n = 256: 79, 50*, 60     n = 512: 170, 93*, 77
  //     B = 16, n = 64: 44*, 47, 77     n = 128: 56, 58*, 82   n = 256: 100, 70*, 97
  //     B = 16, n = 1024: 334, 223*, 212   B = 32, n = 128: 99*, 99, 152   n = 512: 267, 210*, 257
  //   64 rows of 64 tokens   B = 8, n = 128: 175, 103*, 104  n = 512: 560, 298*, 258
  //     B = 16, n = 64: 103*, 104, 146  n = 256: 317, 255*, 291        n = 512: 613, 514*, 468
  //     B = 20, n = 128: 204*, 183, 229 B = 32, n = 128: 332*, 304, 376   n = 256: 516, 455*, 535
  const ClusterFit* fit;
  if (cudaError_t e = g_fits<R, kMulti>.get(L.device, reinterpret_cast<const void*>(cache_attn_tc_kernel<R, kMulti>),
                                            TcCfg<R, kMulti>::kThreads, TcCfg<R, kMulti>::kSmem, &fit))
    return e;
  const long long heads = static_cast<long long>(L.B) * L.H_kv;
  int cs = 1, i = 0;
  while (cs < kMaxCluster && cs * 16 <= L.c.max_pages) {
    const int runs = fit->n[i + 1];
    const long long worth = kMulti ? 64 : 128;         // pages of two blocks, for one wave
    if (heads > runs && (cs > 1 || heads * worth > static_cast<long long>(L.c.max_pages) * runs)) break;
    cs *= 2;
    ++i;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cs, L.H_kv, L.B);
  cfg.blockDim = dim3(TcCfg<R, kMulti>::kThreads);
  cfg.dynamicSmemBytes = TcCfg<R, kMulti>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_tc_kernel<R, kMulti>, L);
}

}  // namespace

cudaError_t launch_cache_attn_tc(const CacheAttnLaunch& L, cudaStream_t st) {
  const int rows = L.H / L.H_kv * L.n;
  if (L.n == 1) return rows <= 32 ? launch<32, false>(L, st) : launch<64, false>(L, st);
  return rows <= 32 ? launch<32, true>(L, st) : launch<64, true>(L, st);
}

}  // namespace focus
