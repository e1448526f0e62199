// The second launch of the verify call over a block-scaled cache: folds a row's
// partials over its prefix pieces (block_stream_kernel) and its draft keys, and
// writes the row.
//
// With (lse, o) of each piece in base 2 the row is sum 2^(lse - m) o / sum
// 2^(lse - m); a draft key counts as a piece of one key.  A warp takes one packed
// row, lane l the columns D / 32 l on, so a piece's row is one coalesced load and
// nothing is computed twice.  SPLIT: the four warps of a CTA share a row's pieces (a
// segment in many pieces is a long chain of loads: two sequences of 6k keys, 2 KV
// heads of 256, 25.6 us without, 23.6 so; 64 sequences in two pieces each 428 without,
// 449 so).  The drafts need nothing of the stream and come first: the kernel is a
// programmatic dependent of it (in plain stream order 3 to 4 us more a call).  All
// sums are 32-bit.
#pragma once
#include "block_stream.cuh"

namespace vsk {

template <int D, bool SPLIT>
__global__ void __launch_bounds__(128) block_combine_kernel(const __grid_constant__ bk::BkParams p) {
  using namespace bk;
  constexpr int E = D / 32;  // columns of a lane
  constexpr int ROWS = SPLIT ? 1 : 4;  // rows of a CTA
  __shared__ int scan[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per_seg = (p.R + ROWS - 1) / ROWS;
  const long long seg = blockIdx.x / per_seg;
  const int row = static_cast<int>(blockIdx.x - seg * per_seg) * ROWS + (SPLIT ? 0 : warp);
  const int b = static_cast<int>(seg / p.h_kv), h = static_cast<int>(seg - static_cast<long long>(b) * p.h_kv);
  const float NEG_INF = -INFINITY;

  int all = 0, before = 0;
  for (int i = tid; i < p.B; i += 128) {
    int P;
    prefix_len(p, i, P);
    const int n = seg_tiles(P);
    all += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) {
    scan[warp] = all;
    scan[4 + warp] = before;
  }
  __syncthreads();
  if (row >= p.R) return;

  const int qa = __ldg(p.qo + b), qe = __ldg(p.qo + b + 1);
  const bool ok = qa >= 0 && qe - qa == p.L && static_cast<long long>(qa) + p.L <= p.n_rows;
  if (!ok && lane == 0 && row == 0 && h == 0) atomicOr(p.err, kErrBadQoIndptr);
  const long long first = ok ? qa : static_cast<long long>(b) * p.L;
  const int i = row / p.gq, head = h * p.gq + row % p.gq;
  int P;
  prefix_len(p, b, P);
  const int T = seg_tiles(P);
  // draft visibility: causal, or the tree mask's row
  const unsigned char* seen = nullptr;
  if (p.cmask) {
    const long long m0 = p.mindptr64 ? static_cast<const long long*>(p.mindptr)[b]
                                     : static_cast<long long>(static_cast<const int*>(p.mindptr)[b]);
    const long long width = static_cast<long long>(P) + p.L;
    if (m0 >= 0 && m0 <= p.n_mask - p.L * width)
      seen = p.cmask + m0 + i * width + P;
    else if (lane == 0 && row == 0 && h == 0)
      atomicOr(p.err, kErrBadMaskIndptr);
  }

  auto load = [&](const __nv_bfloat16* at, float (&x)[E]) {
#pragma unroll
    for (int w = 0; w < E / 2; ++w) {
      const float2 f = unpack_bf16(ld_u32(at + E * lane + 2 * w));
      x[2 * w] = f.x;
      x[2 * w + 1] = f.y;
    }
  };
  float q[E], acc[E], m = NEG_INF, l = 0.f;
  load(p.q + (first + i) * p.q_s0 + static_cast<long long>(head) * p.q_s1, q);
#pragma unroll
  for (int c = 0; c < E; ++c) acc[c] = 0.f;

  // ---- drafts ----
  const int nd = SPLIT && warp > 0 ? 0 : seen ? p.L : i + 1;  // (by the first warp)
  for (int t0 = 0; t0 < nd; t0 += 4) {
    float sc[4], v[4][E];
    bool vis[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = t0 + u;
      vis[u] = t < nd && (!seen || __ldg(seen + t) != 0);
      sc[u] = 0.f;
      if (vis[u]) {
        float k[E];
        load(p.ke + (first + t) * p.ke_s0 + static_cast<long long>(h) * p.ke_s1, k);
        load(p.ve + (first + t) * p.ve_s0 + static_cast<long long>(h) * p.ve_s1, v[u]);
#pragma unroll
        for (int c = 0; c < E; ++c) sc[u] = fmaf(q[c], k[c], sc[u]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < 4; ++u) sc[u] += __shfl_xor_sync(0xffffffffu, sc[u], o);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float x = sc[u] * p.scale2;
      if (!vis[u] || x == NEG_INF) continue;
      if (x > m) {
        const float a = exp2f(m - x);  // 0 while m is -inf
        l *= a;
#pragma unroll
        for (int c = 0; c < E; ++c) acc[c] *= a;
        m = x;
      }
      const float w = exp2f(x - m);
      l += w;
#pragma unroll
      for (int c = 0; c < E; ++c) acc[c] = fmaf(w, v[u][c], acc[c]);
    }
  }

  // ---- pieces: those of the stream's cut ----
  const int total = (scan[0] + scan[1] + scan[2] + scan[3]) * p.n_hg;
  const int off = (scan[4] + scan[5] + scan[6] + scan[7]) * p.n_hg + h / p.team * T;
  const int W = share_of(p, total);
  const int c0 = off / W, all_pieces = (off + T - 1) / W - c0 + 1;
  constexpr int PARTS = SPLIT ? 4 : 1;
  const int pieces = SPLIT ? (all_pieces - warp + PARTS - 1) / PARTS : all_pieces;  // warp, warp + 4, ...
  // piece i: CTA (c0 + i) team + h % team of the stream
  const long long slot = static_cast<long long>(c0) * p.team + static_cast<long long>(b) * p.h_kv + h;
  const long long step = static_cast<long long>(p.team) * p.rows * PARTS;
  const long long at0 = (slot + (SPLIT ? warp * p.team : 0)) * p.rows + row;
  const float* lse = p.plse + at0;
  const float* po = p.po + at0 * D + E * lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i0 = 0; i0 < pieces; i0 += 32) {
    const int n = min(32, pieces - i0);
    const float x = lane < n ? lse[(i0 + lane) * step] : NEG_INF;
    float mx = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (mx > m) {
      const float a = exp2f(m - mx);
      l *= a;
#pragma unroll
      for (int c = 0; c < E; ++c) acc[c] *= a;
      m = mx;
    }
    const float w = x == NEG_INF ? 0.f : exp2f(x - m);
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l += sum;
    constexpr int U = D == 256 ? 4 : 8;  // pieces in flight
    for (int u0 = 0; u0 < n; u0 += U) {
      float2 v[U][E / 2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* src = po + (i0 + min(u0 + u, n - 1)) * step * D;
#pragma unroll
        for (int c = 0; c < E / 2; ++c) v[u][c] = *reinterpret_cast<const float2*>(src + 2 * c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, (u0 + u) & 31);
        if (u0 + u < n && wu != 0.f) {  // the values of an empty piece were never written
#pragma unroll
          for (int c = 0; c < E / 2; ++c) {
            acc[2 * c] = fmaf(wu, v[u][c].x, acc[2 * c]);
            acc[2 * c + 1] = fmaf(wu, v[u][c].y, acc[2 * c + 1]);
          }
        }
      }
    }
  }
  if constexpr (SPLIT) {
    __shared__ float part[3][D + 2];
    if (warp > 0) {
#pragma unroll
      for (int c = 0; c < E; ++c) part[warp - 1][32 * c + lane] = acc[c];
      if (lane == 0) {
        part[warp - 1][D] = m;
        part[warp - 1][D + 1] = l;
      }
    }
    __syncthreads();
    if (warp > 0) return;
    float mx = m;
#pragma unroll
    for (int w = 0; w < 3; ++w) mx = fmaxf(mx, part[w][D]);
    const float ms = mx == NEG_INF ? 0.f : mx;
    float a = exp2f(m - ms);
    l *= a;
#pragma unroll
    for (int c = 0; c < E; ++c) acc[c] *= a;
#pragma unroll
    for (int w = 0; w < 3; ++w) {
      if (part[w][D + 1] == 0.f) continue;  // (a sum that is NaN is none)
      a = exp2f(part[w][D] - ms);
      l = fmaf(a, part[w][D + 1], l);
#pragma unroll
      for (int c = 0; c < E; ++c) acc[c] = fmaf(a, part[w][32 * c + lane], acc[c]);
    }
  }
  // a row with nothing to see is 0
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* o = p.o + (first + i) * p.o_s0 + static_cast<long long>(head) * p.o_s1 + E * lane;
#pragma unroll
  for (int c = 0; c < E / 2; ++c)
    *reinterpret_cast<uint32_t*>(o + 2 * c) = pack_bf16(acc[2 * c] * inv, acc[2 * c + 1] * inv);
}

}  // namespace vsk
