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
// distributed shared memory, so a pass costs one cluster barrier.  To pack the
// output every warp counts what it keeps of its part of the slice and the
// counts are summed over the block and the cluster; positions from ballots
// then sort the slice into a list (kept, others), which the block copies with
// neighbouring threads on neighbouring outputs.  No atomics on the output, so
// the result is exact and in order.
//
// Bound by the mass rows (4 h_kv bytes a key) and, for short sequences, by the
// five cluster barriers.  Measured: 64 sequences of 8,192 to 32,768 keys cut to
// 4,096, 8 heads: 46 us against 11 us of traffic (each pass waits for the
// cluster's slowest CTA); 4 sequences of 800 to 960 keys cut to 256: 10 us.
#pragma once
#include <cooperative_groups.h>

#include "verify_kernel.cuh"

namespace vsk {
namespace ev {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
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
  int cap;         // keys of a slice kept in shared memory (their integers; as many list entries)
  unsigned* err;
};

__device__ __forceinline__ int seq_len(const EvictParams& p, int b, bool& ok) {
  const int a = __ldg(p.kvp + b), e = __ldg(p.kvp + b + 1);
  ok = a >= 0 && e >= a && static_cast<long long>(e) <= p.n_idx;
  return ok ? e - a : 0;
}

// total of key j as an unsigned integer of the same order (+0 and -0 alike, NaN
// largest); eight heads' loads at a time are in flight
__device__ __forceinline__ unsigned order_key(const EvictParams& p, long long j) {
  float t = 0.f;
  for (int h0 = 0; h0 < p.h_kv; h0 += 8) {
    float x[8];
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h0 + h < p.h_kv) x[h] = __ldg(p.mass + (h0 + h) * p.mass_s0 + j);
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h0 + h < p.h_kv) t = h0 + h == 0 ? x[h] : __fadd_rn(t, x[h]);
  }
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
  __shared__ int2 counts[kMaxCluster];  // per CTA of the cluster: keys surely kept, keys at the threshold
  __shared__ long long scan[2][kWarps];
  __shared__ int sel_bin, sel_left, wsum[2][kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = static_cast<int>(blockIdx.x / C);
  cluster.barrier_arrive();  // completes once every CTA runs: its shared memory may then be written

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
      if (pass == 0) cluster.barrier_wait();
      cluster.sync();
      if (warp < 8) {
        // bin 255 - tid: how many keys lie in the bins above it
        int n = 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          if (c < C) n += *cluster.map_shared_rank(hs + 255 - tid, c);
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
  }

  // ---- how many keys of the slice are surely kept, and how many tie ----
  auto classify = [&](int j, int end, bool& sure, bool& tie) {
    sure = tie = false;
    if (j >= end) return;
    if (j >= old) {
      sure = true;
    } else if (want > 0) {
      const unsigned u = key_at(j);
      sure = u > thr;
      tie = u == thr;
    }
  };
  // counts of keys [c0, c1): of this warp's part [w_lo, w_hi) (whole 32s) in
  // wsum, and summed over the parts before it and over all
  int w_lo, w_hi, sure_b, tie_b, sure_all, tie_all;
  auto count = [&](int c0, int c1) {
    const int part = ((c1 - c0 + kWarps - 1) / kWarps + 31) / 32 * 32;
    w_lo = min(c1, c0 + warp * part);
    w_hi = min(c1, w_lo + part);
    int ns = 0, nt = 0;
    for (int j0 = w_lo; j0 < w_hi; j0 += 32) {
      bool sure, tie;
      classify(j0 + lane, w_hi, sure, tie);
      ns += __popc(__ballot_sync(0xffffffffu, sure));
      nt += __popc(__ballot_sync(0xffffffffu, tie));
    }
    if (lane == 0) {
      wsum[0][warp] = ns;
      wsum[1][warp] = nt;
    }
    __syncthreads();
    sure_b = tie_b = sure_all = tie_all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sure_b += w < warp ? wsum[0][w] : 0;
      tie_b += w < warp ? wsum[1][w] : 0;
      sure_all += wsum[0][w];
      tie_all += wsum[1][w];
    }
  };
  count(lo, hi);
  // every CTA hands its counts to all
  if (want <= 0) cluster.barrier_wait();
  if (tid < C) *cluster.map_shared_rank(counts + rank, tid) = make_int2(sure_all, tie_all);
  cluster.sync();
  {
    int s = 0, t = 0;
    for (int c = 0; c < rank; ++c) {
      s += counts[c].x;
      t += counts[c].y;
    }
    const int k = s + min(t, eq_left);  // kept of the sequence before this slice
    kept_before += k;
    gone_before += lo - k;
    eq_left -= min(t, eq_left);
  }

  // ---- pack, cap keys at a time: positions into a list (the kept ones, then
  // the others), which the whole block then copies, neighbours by neighbours ----
  unsigned* list = keys + p.cap;
  for (int c0 = lo; c0 < hi; c0 += p.cap) {
    const int n = min(p.cap, hi - c0);
    if (n < hi - lo) {  // (a single chunk was counted above)
      __syncthreads();
      count(c0, c0 + n);
    }
    const int kept_n = sure_all + min(tie_all, eq_left);
    int k0 = sure_b + min(tie_b, eq_left), left = eq_left - min(tie_b, eq_left);
    for (int j0 = w_lo; j0 < w_hi; j0 += 32) {
      const int j = j0 + lane;
      bool sure, tie;
      classify(j, w_hi, sure, tie);
      const unsigned ms = __ballot_sync(0xffffffffu, sure), mt = __ballot_sync(0xffffffffu, tie);
      const unsigned below = (1u << lane) - 1u;
      const int t_b = __popc(mt & below), at = k0 + __popc(ms & below) + min(t_b, left);
      if (j < w_hi) list[(sure || (tie && t_b < left)) ? at : kept_n + (j - c0) - at] = static_cast<unsigned>(j);
      k0 += __popc(ms) + min(__popc(mt), left);
      left -= min(__popc(mt), left);
    }
    __syncthreads();
#pragma unroll 2
    for (int i = tid; i < n; i += kThreads) {
      const bool keep = i < kept_n;
      const long long from = kv0 + list[i], to = keep ? kept_before + i : gone_before + i - kept_n;
      if (to < (keep ? p.out_cap : p.freed_cap)) copy_index(p, keep ? p.out_idx : p.freed, to, from);
    }
    for (int i = tid; i < kept_n; i += kThreads) {
      const long long from = kv0 + list[i], to = kept_before + i;
      if (to >= p.out_cap) break;
      for (int h0 = 0; h0 < p.h_kv; h0 += 8) {
        float x[8];
#pragma unroll
        for (int h = 0; h < 8; ++h)
          if (h0 + h < p.h_kv) x[h] = __ldg(p.mass + (h0 + h) * p.mass_s0 + from);
#pragma unroll
        for (int h = 0; h < 8; ++h)
          if (h0 + h < p.h_kv) p.out_mass[(h0 + h) * p.out_s0 + to] = x[h];
      }
    }
    kept_before += kept_n;
    gone_before += n - kept_n;
    eq_left -= min(tie_all, eq_left);
  }
}

}  // namespace vsk
