// kv_evict: cuts every sequence's cache index down to `budget` entries by
// accumulated attention weight.
//
// A sequence of at most `budget` keys keeps them all.  A longer one keeps its
// last `recent` keys and, of the others, the budget - recent with the largest
//   total[j] = mass[0][j] + mass[1][j] + ...   (32-bit, heads in ascending order)
// (equal totals: the lowest positions; NaN counts as the largest), in their
// order.  The kept indices and mass columns are written packed, the indices
// of the others go to `freed`, both sequence after sequence.
//
// The k-th largest total is found by radix selection: totals map to unsigned
// integers of the same order, and four passes of 8 bits narrow down the k-th
// one by counting.  One thread-block cluster owns a sequence; each CTA keeps its
// slice's integers in shared memory (mass is read once; what does not fit is
// summed again), counts into a 256-bin histogram and reads the others' through
// distributed shared memory, so a pass costs one cluster barrier.  A second
// walk over the slice packs the output: positions come from ballots and a scan
// over the block, no atomics, so the result is exact and in order.
//
// Bound by the mass rows (4 h_kv bytes a key) and, for short sequences, by the
// seven cluster barriers.
#pragma once
#include <cooperative_groups.h>

#include "verify_kernel.cuh"

namespace vsk {
namespace ev {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kErrNoRoom = 32u;  // an output is shorter than what is written to it

struct EvictParams {
  const float* mass; long long mass_s0;
  const int* kvp;
  const void* kvi;
  int idx64, h_kv, B;
  long long n_idx, budget, recent;
  int* out_ptr;
  void* out_idx;   // of kvi's type
  float* out_mass; long long out_s0;
  void* freed;     // of kvi's type
  long long out_cap, freed_cap;
  int cap;         // integers of a slice kept in shared memory
  unsigned* err;
};

__device__ __forceinline__ int seq_len(const EvictParams& p, int b, bool& ok) {
  const int a = __ldg(p.kvp + b), e = __ldg(p.kvp + b + 1);
  ok = a >= 0 && e >= a && static_cast<long long>(e) <= p.n_idx;
  return ok ? e - a : 0;
}

// total of key j as an unsigned integer of the same order (+0 and -0 alike, NaN largest)
__device__ __forceinline__ unsigned order_key(const EvictParams& p, long long j) {
  float t = __ldg(p.mass + j);
  for (int h = 1; h < p.h_kv; ++h) t = __fadd_rn(t, __ldg(p.mass + h * p.mass_s0 + j));
  if (t != t) return 0xFFFFFFFFu;
  const unsigned u = __float_as_uint(t + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void copy_index(const EvictParams& p, void* dst, long long at, long long from) {
  if (p.idx64)
    static_cast<long long*>(dst)[at] = __ldg(static_cast<const long long*>(p.kvi) + from);
  else
    static_cast<int*>(dst)[at] = __ldg(static_cast<const int*>(p.kvi) + from);
}

}  // namespace ev

__global__ void __launch_bounds__(ev::kThreads) evict_kernel(const __grid_constant__ ev::EvictParams p) {
  using namespace ev;
  namespace cg = cooperative_groups;
  extern __shared__ unsigned keys[];
  __shared__ int hist[2][256];
  __shared__ int counts[2];             // this CTA's keys above the threshold, and at it
  __shared__ long long scan[2][kWarps];
  __shared__ int sel_bin, sel_left, wsum[2][kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = static_cast<int>(blockIdx.x / C);

  // ---- where this sequence's output starts ----
  long long kept_before = 0, gone_before = 0;
  for (int i = tid; i < b; i += kThreads) {
    bool ok;
    const long long n = seq_len(p, i, ok), k = min(n, p.budget);
    kept_before += k;
    gone_before += n - k;
  }
  kept_before = warp_sum(kept_before);
  gone_before = warp_sum(gone_before);
  if (lane == 0) {
    scan[0][warp] = kept_before;
    scan[1][warp] = gone_before;
  }
  __syncthreads();
  kept_before = gone_before = 0;
  for (int w = 0; w < kWarps; ++w) {
    kept_before += scan[0][w];
    gone_before += scan[1][w];
  }
  bool ok;
  const int P = seq_len(p, b, ok);
  const long long kv0 = ok ? __ldg(p.kvp + b) : 0;
  const bool select = P > p.budget;
  const int kept = static_cast<int>(min(static_cast<long long>(P), p.budget));
  const int old = select ? static_cast<int>(P - p.recent) : 0;  // keys [0, old) are chosen from
  if (rank == 0 && tid == 0) {
    if (!ok) atomicOr(p.err, kErrBadKvIndptr);
    if (kept_before + kept > p.out_cap || gone_before + P - kept > p.freed_cap) atomicOr(p.err, kErrNoRoom);
    if (b == 0) p.out_ptr[0] = 0;
    p.out_ptr[b + 1] = static_cast<int>(kept_before + kept);
  }
  const int per = (P + C - 1) / C;
  const int lo = static_cast<int>(min(static_cast<long long>(P), static_cast<long long>(rank) * per));
  const int hi = min(P, lo + per);
  const int lo_o = min(lo, old), hi_o = min(hi, old);  // the slice's part of [0, old)
  auto key_at = [&](int j) -> unsigned { return j - lo < p.cap ? keys[j - lo] : order_key(p, kv0 + j); };

  // ---- the threshold: the (budget - recent)-th largest key of [0, old) ----
  unsigned thr = 0xFFFFFFFFu;
  int eq_left = 0;  // keys at the threshold that are kept, lowest positions first
  const int want = select ? static_cast<int>(p.budget - p.recent) : 0;
  if (want > 0) {  // uniform over the cluster
    for (int j = lo_o + tid; j < min(hi_o, lo + p.cap); j += kThreads) keys[j - lo] = order_key(p, kv0 + j);
    unsigned prefix = 0u, mask = 0u;
    int k = want;  // still to be found among the keys that match the prefix
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      int* hs = hist[pass & 1];
      for (int i = tid; i < 256; i += kThreads) hs[i] = 0;
      __syncthreads();  // also: keys are complete
      for (int j = lo_o + tid; j < hi_o; j += kThreads) {
        const unsigned u = key_at(j);
        if ((u & mask) == prefix) atomicAdd(hs + ((u >> shift) & 255u), 1);
      }
      cluster.sync();
      if (warp < 8) {
        // bin 255 - tid: how many keys lie in the bins above it
        int n = 0;
        for (int c = 0; c < C; ++c) n += *cluster.map_shared_rank(hs + 255 - tid, c);
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (lane == 31) wsum[0][warp] = incl;
        named_bar_sync(1, 256);
        for (int w = 0; w < warp; ++w) incl += wsum[0][w];
        if (incl >= k && incl - n < k) {
          sel_bin = 255 - tid;
          sel_left = k - (incl - n);
        }
      }
      __syncthreads();
      prefix |= static_cast<unsigned>(sel_bin) << shift;
      mask |= 255u << shift;
      k = sel_left;
    }
    thr = prefix;
    eq_left = k;
    // ---- keys above and at the threshold in the slices before this one ----
    int gt = 0, eq = 0;
    for (int j = lo_o + tid; j < hi_o; j += kThreads) {
      const unsigned u = key_at(j);
      gt += u > thr;
      eq += u == thr;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (tid == 0) counts[0] = counts[1] = 0;
    __syncthreads();
    if (lane == 0) {
      atomicAdd(counts, gt);
      atomicAdd(counts + 1, eq);
    }
    cluster.sync();
    int gt_b = 0, eq_b = 0;
    for (int c = 0; c < rank; ++c) {
      gt_b += *cluster.map_shared_rank(counts, c);
      eq_b += *cluster.map_shared_rank(counts + 1, c);
    }
    const int eq_k = min(eq_left, eq_b);
    const int kept_o = gt_b + eq_k;
    kept_before += kept_o + (lo - lo_o);
    gone_before += lo_o - kept_o;
    eq_left -= eq_k;
    cluster.sync();  // the counts have been read
  } else {
    // nothing of [0, old) is kept
    kept_before += lo - lo_o;
    gone_before += lo_o;
  }

  // ---- pack the slice ----
  for (int j0 = lo; j0 < hi; j0 += kThreads) {
    const int j = j0 + tid;
    bool sure = false, tie = false;
    if (j < hi) {
      if (j >= old) {
        sure = true;
      } else if (want > 0) {
        const unsigned u = key_at(j);
        sure = u > thr;
        tie = u == thr;
      }
    }
    const unsigned ms = __ballot_sync(0xffffffffu, sure), mt = __ballot_sync(0xffffffffu, tie);
    __syncthreads();  // the sums of the round before have been read
    if (lane == 0) {
      wsum[0][warp] = __popc(ms);
      wsum[1][warp] = __popc(mt);
    }
    __syncthreads();
    const unsigned below = (1u << lane) - 1u;
    int s_b = __popc(ms & below), t_b = __popc(mt & below), s_all = 0, t_all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        s_b += wsum[0][w];
        t_b += wsum[1][w];
      }
      s_all += wsum[0][w];
      t_all += wsum[1][w];
    }
    const bool keep = sure || (tie && t_b < eq_left);
    const int before = s_b + min(t_b, eq_left);  // kept keys before j in this round
    if (j < hi) {
      if (keep) {
        const long long at = kept_before + before;
        if (at < p.out_cap) {
          copy_index(p, p.out_idx, at, kv0 + j);
          for (int h = 0; h < p.h_kv; ++h) p.out_mass[h * p.out_s0 + at] = __ldg(p.mass + h * p.mass_s0 + kv0 + j);
        }
      } else {
        const long long at = gone_before + tid - before;
        if (at < p.freed_cap) copy_index(p, p.freed, at, kv0 + j);
      }
    }
    const int n = min(kThreads, hi - j0), k = s_all + min(t_all, eq_left);
    kept_before += k;
    gone_before += n - k;
    eq_left -= min(t_all, eq_left);
  }
}

}  // namespace vsk
