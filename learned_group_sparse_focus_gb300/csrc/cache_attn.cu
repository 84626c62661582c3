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
#include "cache_attn.cuh"

namespace focus {
namespace {

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
